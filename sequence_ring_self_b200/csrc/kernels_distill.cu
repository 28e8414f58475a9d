// kernels_distill.cu -- distillation from a teacher's top logits: loss, gradient, or both in
// one pass (rsa_distill*, rsa_rows.h).
//
//   p = softmax(teacher / tau) over a row's live slots,  q = softmax(z / tau) over its V logits
//   loss = tau^2 sum_j p_j (ln p_j - ln q_{index_j}),    dz = dloss tau (q - p)
//
// Bound by memory (a row is V elements read, and V written by the gradient), with the exponent
// unit close behind: one exponential per element and pass. CTAs are persistent and take rows in
// turn; a row belongs to one CTA, or to a cluster that shares its columns where there are few
// rows or one CTA cannot hold it. Every thread keeps a running maximum and sum of exponentials of
// the 16-byte vectors it reads; the CTA joins them by shuffles and the cluster through
// distributed shared memory, always in the same order. The gradient is streamed as dloss tau q,
// and the few columns with a teacher's slot are written once more afterwards, from logits read
// before anything of the row was written (which lets the gradient replace the logits in place).
// One block barrier per row: it makes the row's sums whole, the last row's slots visible, and
// tells whether the next row has a slot at all. Nothing of a row without one is used, but a CTA's
// first row, and in one pass the beginning of every next row, is sent for before that is known.
#include <cooperative_groups.h>
#include <type_traits>

#include "rows_common.cuh"

namespace rsa {
namespace {

using namespace rows;
namespace cg = cooperative_groups;

constexpr int kPassBatch = 2;  // vectors of a thread's batch
constexpr int kRing = 4;       // batches of a thread on their way
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// 2^x by the hardware's approximation (about 2 units in the last place). Results below the
// smallest normal number flush to zero: a probability below 2^-126 adds nothing to a sum that
// is at least 1, and rounds to no bf16 or fp32 gradient that matters next to it.
__device__ __forceinline__ float exp2_ftz(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Running maximum m and s = sum 2^((z - m) c). Differences are taken before the scaling: they are
// exact where it matters, and a logit of the type's lowest value cannot overflow against another
// of the same.
struct MaxSum {
    float m, s;
};

__device__ __forceinline__ MaxSum join(MaxSum a, MaxSum b, float c) {
    const float m = fmaxf(a.m, b.m);
    // nothing but -infinity (or NaN) so far: the sums are 0 (or NaN) and stay so
    const float ref = m == -INFINITY ? 0.f : m;
    // products and sum rounded one by one, so that join(a, b) = join(b, a) and a butterfly of
    // shuffles leaves the same bits in every lane
    return {m, __fadd_rn(__fmul_rn(a.s, exp2_ftz((a.m - ref) * c)),
                         __fmul_rn(b.s, exp2_ftz((b.m - ref) * c)))};
}

// The pairs of LANES neighbouring lanes, as one: the maximum first, then the sums brought to it.
template <int LANES>
__device__ __forceinline__ MaxSum join_lanes(MaxSum r, float c) {
    float m = r.m;
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float s = r.s * exp2_ftz((r.m - (m == -INFINITY ? 0.f : m)) * c);
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return {m, s};
}

// The pairs that W warps have left, as one.
template <int W>
__device__ __forceinline__ MaxSum join_warps(const float2 (&part)[W], float c) {
    const int lane = threadIdx.x & 31;
    constexpr int N = W <= 1 ? 1 : W <= 2 ? 2 : W <= 4 ? 4 : W <= 8 ? 8 : W <= 16 ? 16 : 32;
    const float2 v = (lane & (N - 1)) < W ? part[lane & (N - 1)] : make_float2(-INFINITY, 0.f);
    return join_lanes<N>({v.x, v.y}, c);
}

// A thread's share of a row, with the sum in four parts.
struct Running {
    float m;
    float2 s[2];

    __device__ __forceinline__ float ref() const { return m == -INFINITY ? 0.f : m; }
    __device__ __forceinline__ void raise(float to, float c) {
        if (to > m) {
            const float2 f = both(exp2_ftz((m - to) * c));
            s[0] = mul2(s[0], f);
            s[1] = mul2(s[1], f);
            m = to;
        }
    }
    __device__ __forceinline__ void one(float z, float c) {
        raise(z, c);
        s[0].x += exp2_ftz((z - ref()) * c);
    }
    __device__ __forceinline__ MaxSum sum() const {
        return {m, (s[0].x + s[0].y) + (s[1].x + s[1].y)};
    }
};

// The largest of a batch of vectors; bf16 is compared two at a time.
template <typename T, int N, typename P>
__device__ __forceinline__ float largest(const P (&v)[N]) {
    if constexpr (sizeof(T) == 2) {
        auto pair = [](uint32_t w) { return *reinterpret_cast<__nv_bfloat162 *>(&w); };
        __nv_bfloat162 m = pair(v[0].raw.x);
#pragma unroll
        for (int i = 0; i < N; ++i)
            m = __hmax2(m, __hmax2(__hmax2(pair(v[i].raw.x), pair(v[i].raw.y)),
                                   __hmax2(pair(v[i].raw.z), pair(v[i].raw.w))));
        return fmaxf(__low2float(m), __high2float(m));
    } else {
        float m = -INFINITY;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float f[4];
            v[i].to(f);
            m = fmaxf(fmaxf(m, fmaxf(f[0], f[1])), fmaxf(f[2], f[3]));
        }
        return m;
    }
}

// What a CTA of NT threads, U vectors per thread and batch, knows of its share of the rows.
template <typename T, int NT, int U>
struct Rows {
    static constexpr int VEC = 16 / sizeof(T), E = VEC / 2, W = NT / 32, STEP = NT * U;
    static constexpr uint32_t kNone = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;  // -infinity
    using P = Pack<T, VEC>;

    const DistillArgs &a;
    int rank, nc, Kp;  // CTA of the cluster; slots rounded up to a multiple of four
    uint4 *mine;       // the thread's places for batches: vector u of batch b at (b U + u) NT
    int *lists;        // places of [index][teacher logit, then probability][student logit] x Kp
    float c;

    // The CTA's columns of a row: `head` single elements up to the first 16-byte boundary (rank
    // 0), n vectors from zv on, and single elements behind the last vector (the last rank). The
    // vectors come in nb batches; the first one has n0 of them, the others U per thread, so
    // that their loop has neither conditions nor address arithmetic.
    struct Share {
        const T *z, *zv;
        int head, tail, first, n, n0, nb;
    };
    __device__ __forceinline__ Share share_of(int row) const {
        Share s;
        s.z = static_cast<const T *>(a.z) + row * a.ld;
        const int mis = static_cast<int>(reinterpret_cast<uintptr_t>(s.z) / sizeof(T)) & (VEC - 1);
        s.head = min(a.V, mis ? VEC - mis : 0);
        const int nv = (a.V - s.head) / VEC, per = (nv + nc - 1) >> a.log_cluster;
        s.tail = s.head + nv * VEC;
        const int v0 = min(nv, rank * per);
        s.n = min(nv - v0, per);
        s.first = s.head + v0 * VEC;
        s.zv = s.z + s.first;
        s.nb = (s.n + STEP - 1) / STEP;
        s.n0 = s.n - max(s.nb - 1, 0) * STEP;
        return s;
    }
    __device__ __forceinline__ int low(const Share &s) const { return rank ? s.first : 0; }
    __device__ __forceinline__ int high(const Share &s) const {
        return rank == nc - 1 ? a.V : s.first + s.n * VEC;
    }
    __device__ __forceinline__ bool has_head(const Share &s) const {
        return rank == 0 && static_cast<int>(threadIdx.x) < s.head;
    }
    __device__ __forceinline__ bool has_tail(const Share &s) const {
        return rank == nc - 1 && static_cast<int>(threadIdx.x) < a.V - s.tail;
    }
    // The thread's first vector behind the first batch; batch b > 0 lies (b - 1) STEP vectors on.
    __device__ __forceinline__ const T *behind_first(const Share &s) const {
        return s.zv + (s.n0 + static_cast<int>(threadIdx.x)) * VEC;
    }
    // A batch on its way to the thread's places: the first one, or one from p on.
    __device__ __forceinline__ void fetch_first(const Share &s, uint4 *to) const {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int at = threadIdx.x + u * NT;
            if (at < s.n0) cp_async16(to + u * NT, s.zv + at * VEC);
        }
    }
    __device__ __forceinline__ static void fetch(const T *p, uint4 *to) {
#pragma unroll
        for (int u = 0; u < U; ++u) cp_async16(to + u * NT, p + u * NT * VEC);
    }
    __device__ __forceinline__ static void take(const uint4 *from, P (&v)[U]) {
#pragma unroll
        for (int u = 0; u < U; ++u) v[u].raw = from[u * NT];
    }
    // -infinity behind the end of a first batch.
    __device__ __forceinline__ void fill(const Share &s, P (&v)[U]) const {
        if (s.n0 < STEP) {
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (static_cast<int>(threadIdx.x) + u * NT >= s.n0)
                    v[u].raw = make_uint4(kNone, kNone, kNone, kNone);
        }
    }
    // The first kRing batches of a row, a group each, whether or not there is any.
    __device__ __forceinline__ void fetch_ring(const Share &s) const {
        fetch_first(s, mine);
        cp_async_commit();
#pragma unroll
        for (int b = 1; b < kRing; ++b) {
            if (b < s.nb) fetch(behind_first(s) + (b - 1) * STEP * VEC, mine + b * STEP);
            cp_async_commit();
        }
    }

    __device__ __forceinline__ void slot_of(int row, int j, int &id, float &x) const {
        const long long at = static_cast<long long>(row) * a.K + j, i = index_at(a.index, a.index64, at);
        x = a.teacher_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(a.teacher)[at])
                           : static_cast<const float *>(a.teacher)[at];
        id = i >= 0 && i < a.V && x != -INFINITY ? static_cast<int>(i) : -1;
    }
    __device__ __forceinline__ float logit_of(int row, int id) const {
        return id >= 0 ? static_cast<float>(static_cast<const T *>(a.z)[row * a.ld + id]) : 0.f;
    }
    __device__ __forceinline__ int *slots(int place) const { return lists + place * 3 * Kp; }
    __device__ __forceinline__ float *probs(int place) const {
        return reinterpret_cast<float *>(slots(place) + Kp);
    }
    __device__ __forceinline__ float *logits(int place) const { return probs(place) + Kp; }
    // A row's slots into the lists: the thread's first, loaded before, and the NTth on. The lists
    // belong to the threads that write them until a barrier.
    __device__ __forceinline__ bool list_slots(int row, int place, int id, float x) const {
        bool live = false;
        for (int j = threadIdx.x; j < Kp; j += NT) {
            if (j >= NT) {
                id = -1, x = -INFINITY;
                if (j < a.K) slot_of(row, j, id, x);
            }
            live |= id >= 0;
            slots(place)[j] = id;
            probs(place)[j] = x;
            logits(place)[j] = logit_of(row, id);
        }
        return live;
    }
    // The thread's part of the teacher's maximum and sum.
    __device__ __forceinline__ MaxSum teacher(int place) const {
        MaxSum t = {-INFINITY, 0.f};
        for (int j = threadIdx.x; j < a.K; j += NT)
            if (slots(place)[j] >= 0) t = join(t, {probs(place)[j], 1.f}, c);
        return t;
    }
    // The thread's slots of a row: probabilities into the lists, and its part of the loss over tau
    // (m, logsum: the row's maximum and log2 of its sum): p (tau (ln p + ln sum) - (z - m)), in which
    // a logit of the type's lowest value is not scaled before its probability has made it small.
    __device__ __forceinline__ float finish_slots(int place, MaxSum t, float m, float logsum) const {
        const float tl2 = log2f(t.s), nat = a.tau * kLn2;
        float l = 0.f;
        for (int j = threadIdx.x; j < Kp; j += NT) {
            const float lp = (probs(place)[j] - t.m) * c - tl2;  // log2 p
            const float p = slots(place)[j] >= 0 ? exp2_ftz(lp) : 0.f;
            if (p != 0.f) l += p * (nat * (lp + logsum) - (logits(place)[j] - m));
            probs(place)[j] = p;
        }
        return l;
    }

    // Adds a batch to the running maximum and sum.
    __device__ __forceinline__ void add(Running &r, const P (&v)[U]) const {
        r.raise(largest<T>(v), c);
        const float2 ref = both(-r.ref()), c2 = both(c);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float2 f[E];
            v[u].to(f);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                f[e] = mul2(add2(f[e], ref), c2);
                r.s[e & 1] = add2(r.s[e & 1], make_float2(exp2_ftz(f[e].x), exp2_ftz(f[e].y)));
            }
        }
    }
    // Runs f(batch, vectors) over a row whose first kRing batches are on their way; each place is
    // refilled when it is used up.
    template <typename F>
    __device__ __forceinline__ void stream(const Share &s, F &&f) const {
        const T *p = behind_first(s) + (kRing - 1) * STEP * VEC;
        int place = 0;
        for (int b = 0; b < s.nb; ++b, p += STEP * VEC) {
            P v[U];
            cp_async_wait<kRing - 1>();
            take(mine + place, v);
            f(b, v);
            if (b + kRing < s.nb) fetch(p, mine + place);
            cp_async_commit();
            place = place == (kRing - 1) * STEP ? 0 : place + STEP;
        }
        cp_async_wait<0>();
    }
    // Runs f(batch, vectors) over the batches [b, end), b > 0, straight from memory, one ahead.
    template <typename F>
    __device__ __forceinline__ void walk(const Share &s, int b, int end, F &&f) const {
        if (b >= end) return;
        const T *p = behind_first(s) + (b - 1) * static_cast<long long>(STEP * VEC);
        P v[U], w[U];
        load(p, v);
        for (;; b += 2, p += 2 * STEP * VEC) {
            if (b + 1 < end) load(p + STEP * VEC, w);
            f(b, v);
            if (b + 1 >= end) break;
            if (b + 2 < end) load(p + 2 * STEP * VEC, v);
            f(b + 1, w);
            if (b + 2 >= end) break;
        }
    }
    __device__ __forceinline__ static void load(const T *p, P (&v)[U]) {
#pragma unroll
        for (int u = 0; u < U; ++u) v[u] = P::load(p + u * NT * VEC);
    }
    __device__ __forceinline__ void add_ends(const Share &s, Running &r) const {
        if (has_head(s)) r.one(static_cast<float>(s.z[threadIdx.x]), c);
        if (has_tail(s)) r.one(static_cast<float>(s.z[s.tail + threadIdx.x]), c);
    }
};

// One row's gradient g (q - p): g = dloss tau, m and logsum its maximum and log2 of its sum.
template <typename T, int NT, int U>
struct Gradient {
    using R = Rows<T, NT, U>;
    using Share = typename R::Share;
    using P = typename R::P;
    T *dz;
    float m, logsum, g;

    __device__ __forceinline__ Gradient(const R &rows, int row, float m, float logsum)
        : dz(static_cast<T *>(rows.a.dz) + row * rows.a.ld_d), m(m), logsum(logsum),
          g(rows.a.dloss[row * rows.a.dloss_stride] * rows.a.tau) {}
    __device__ __forceinline__ float of(const R &rows, float z, float p) const {
        return g * (exp2_ftz((z - m) * rows.c - logsum) - p);
    }
    template <bool ALIGNED>
    __device__ __forceinline__ void vector(const R &rows, T *to, const P &v) const {
        float2 f[R::E];
        v.to(f);
#pragma unroll
        for (int e = 0; e < R::E; ++e) {
            f[e] = fma2(add2(f[e], both(-m)), both(rows.c), both(-logsum));
            f[e] = mul2(both(g), make_float2(exp2_ftz(f[e].x), exp2_ftz(f[e].y)));
        }
        if (ALIGNED) {
            // written once and not read here again: first to leave L2
            __stcs(reinterpret_cast<uint4 *>(to), P::from(f).raw);
        } else {
#pragma unroll
            for (int e = 0; e < R::E; ++e) to[2 * e] = T(f[e].x), to[2 * e + 1] = T(f[e].y);
        }
    }
    __device__ __forceinline__ bool aligned(const Share &s) const {
        return ((reinterpret_cast<uintptr_t>(s.z) ^ reinterpret_cast<uintptr_t>(dz)) & 15u) == 0;
    }
    // Batch b of the row: vectors where those of the logits are vectors of the gradient, else
    // element by element.
    __device__ __forceinline__ void batch(const R &rows, const Share &s, int b, bool vec,
                                          const P (&v)[U]) const {
        if (b == 0) {
            T *to = dz + s.first + static_cast<int>(threadIdx.x) * R::VEC;
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (static_cast<int>(threadIdx.x) + u * NT < s.n0) {
                    if (vec)
                        vector<true>(rows, to + u * NT * R::VEC, v[u]);
                    else
                        vector<false>(rows, to + u * NT * R::VEC, v[u]);
                }
        } else {
            T *to = dz + s.first +
                    static_cast<long long>(s.n0 + static_cast<int>(threadIdx.x) + (b - 1) * R::STEP) * R::VEC;
            if (vec)
                full<true>(rows, to, v);
            else
                full<false>(rows, to, v);
        }
    }
    template <bool ALIGNED>
    __device__ __forceinline__ void full(const R &rows, T *to, const P (&v)[U]) const {
#pragma unroll
        for (int u = 0; u < U; ++u) vector<ALIGNED>(rows, to + u * NT * R::VEC, v[u]);
    }
    __device__ __forceinline__ void ends(const R &rows, const Share &s) const {
        if (rows.has_head(s)) dz[threadIdx.x] = T(of(rows, static_cast<float>(s.z[threadIdx.x]), 0.f));
        if (rows.has_tail(s))
            dz[s.tail + threadIdx.x] = T(of(rows, static_cast<float>(s.z[s.tail + threadIdx.x]), 0.f));
    }
    // The columns that a slot points to, from the lists (those with the same index add up).
    __device__ __forceinline__ void columns(const R &rows, const Share &s, int place) const {
        const int low = rows.low(s), high = rows.high(s);
        const int *slot = rows.slots(place);
        const float *prob = rows.probs(place), *zs = rows.logits(place);
        for (int j = threadIdx.x; j < rows.a.K; j += NT) {
            const int id = slot[j];
            if (id < low || id >= high) continue;
            float p = 0.f;
            for (int i = 0; i < rows.Kp; i += 4) {
                const int4 n = *reinterpret_cast<const int4 *>(slot + i);
                const float4 w = *reinterpret_cast<const float4 *>(prob + i);
                p += n.x == id ? w.x : 0.f;
                p += n.y == id ? w.y : 0.f;
                p += n.z == id ? w.z : 0.f;
                p += n.w == id ? w.w : 0.f;
            }
            dz[id] = T(of(rows, zs[j], p));
        }
    }
    __device__ __forceinline__ void zeros(const R &rows, const Share &s) const {
        // counted without a sign: a share may end within NT of 2^31
        T *to = dz + rows.low(s);
        const unsigned count = rows.high(s) - rows.low(s);
        for (unsigned j = threadIdx.x; j < count; j += NT) to[j] = T(0.f);
    }
};

enum { kForward, kBackward, kStep };
constexpr int kPlaces = 4;  // rows whose lists are in use between two barriers, and one more

// Sum of the warps' parts of a row's loss over tau, as the loss.
template <int W>
__device__ __forceinline__ float row_loss(const float (&part)[W], float tau) {
    float l = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) l += part[w];
    return tau * l;
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// A row's pair over its CTAs, by distributed shared memory (two places in turn: a pair is not
// replaced before the next row's barrier, which its readers have passed by then).
__device__ __forceinline__ MaxSum join_cluster(MaxSum q, float2 *place, int nc, float c) {
    cg::cluster_group cluster = cg::this_cluster();
    if (threadIdx.x == 0) *place = make_float2(q.m, q.s);
    cluster.sync();
    q = {-INFINITY, 0.f};
    for (int k = 0; k < nc; ++k) {
        const float2 o = *cluster.map_shared_rank(place, k);
        q = join(q, {o.x, o.y}, c);
    }
    return q;
}

// A row's maximum, and log2 of its sum, where it holds a NaN or nothing but -infinity.
__device__ __forceinline__ float log_of(MaxSum q, float &m) {
    m = q.s != q.s && q.m != INFINITY ? q.s : q.m;
    return m == -INFINITY ? NAN : log2f(q.s);
}

// Loss and statistics, or the gradient from them.
template <typename T, bool BACKWARD, int NT>
__global__ void __launch_bounds__(NT, 1024 / NT) distill_kernel(const DistillArgs a) {
    constexpr int U = kPassBatch;
    using R = Rows<T, NT, U>;
    using P = typename R::P;
    constexpr int W = R::W;
    extern __shared__ __align__(16) uint4 dyn[];
    __shared__ float2 red_row[2][W], red_slots[2][W], shared_ms[2];
    __shared__ float red_loss[2][W];
    pdl_wait();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int nc = 1 << a.log_cluster;
    const R rows = {a, static_cast<int>(cg::this_cluster().block_rank()), nc, (a.K + 3) & ~3,
                    dyn + tid, reinterpret_cast<int *>(dyn + kRing * R::STEP), kLog2e / a.tau};
    const float c = rows.c;

    const int stride = gridDim.x >> a.log_cluster;
    int row = blockIdx.x >> a.log_cluster, par = 0, place = 0, last_row = -1;
    bool alive;
    {
        int id = -1;
        float x = -INFINITY;
        if (tid < a.K) rows.slot_of(row, tid, id, x);
        rows.fetch_ring(rows.share_of(row));  // whether or not the first row has a slot
        const bool live = rows.list_slots(row, 0, id, x);
        if (BACKWARD) {
            const MaxSum t = join_lanes<32>(rows.teacher(0), c);
            if (lane == 0) red_slots[1][warp] = make_float2(t.m, t.s);
        }
        alive = __syncthreads_or(live);
        if (!alive) cp_async_wait<0>();
        if (BACKWARD) rows.finish_slots(0, join_warps(red_slots[1], c), 0.f, 0.f);
    }

    for (; row < a.n; row += stride, par ^= 1) {
        const int next_row = row + stride;
        const bool has_next = next_row < a.n;
        int next_id = -1;
        float next_x = -INFINITY;
        if (has_next && tid < a.K) rows.slot_of(next_row, tid, next_id, next_x);
        Running r = {-INFINITY, {make_float2(0.f, 0.f), make_float2(0.f, 0.f)}};
        const typename R::Share cur = rows.share_of(row);
        if (BACKWARD) {
            const float2 st = static_cast<const float2 *>(a.stats)[row];
            const Gradient<T, NT, U> grad(rows, row, st.x, st.y * kLog2e);
            if (alive) {
                grad.ends(rows, cur);
                const bool vec = grad.aligned(cur);
                rows.stream(cur, [&](int b, P(&v)[U]) { grad.batch(rows, cur, b, vec, v); });
            } else {
                grad.zeros(rows, cur);
            }
        } else if (alive) {
            rows.add_ends(cur, r);
            rows.stream(cur, [&](int b, P(&v)[U]) {
                if (b == 0) rows.fill(cur, v);
                rows.add(r, v);
            });
        }

        // the next row's slots and their logits, read before anything of that row is replaced
        const int next_place = (place + 1) % kPlaces;
        bool live = false;
        if (has_next) live = rows.list_slots(next_row, next_place, next_id, next_x);
        // pairs of the warps: the row's and its teacher's, or the next row's teacher's
        MaxSum t = {-INFINITY, 0.f}, q = t;
        if (!BACKWARD || has_next)
            t = join_lanes<32>(rows.teacher(BACKWARD ? next_place : place), c);
        if (!BACKWARD) q = join_lanes<32>(r.sum(), c);
        if (lane == 0) {
            red_row[par][warp] = make_float2(q.m, q.s);
            red_slots[par][warp] = make_float2(t.m, t.s);
        }
        const bool next_alive = __syncthreads_or(live);
        if (next_alive) rows.fetch_ring(rows.share_of(next_row));
        t = join_warps(red_slots[par], c);
        if (BACKWARD) {
            if (alive) {
                const float2 st = static_cast<const float2 *>(a.stats)[row];
                Gradient<T, NT, U>(rows, row, st.x, st.y * kLog2e).columns(rows, cur, place);
            }
            if (has_next) rows.finish_slots(next_place, t, 0.f, 0.f);
        } else {
            // the last row's loss, its parts complete since this barrier
            if (last_row >= 0 && rows.rank == 0 && tid == 0)
                a.loss[last_row] = row_loss(red_loss[par ^ 1], a.tau);
            q = join_warps(red_row[par], c);
            if (nc > 1) q = join_cluster(q, &shared_ms[par], nc, c);
            float m;
            const float logsum = log_of(q, m);
            const float l = warp_sum(rows.finish_slots(place, t, m, logsum));
            if (lane == 0) red_loss[par][warp] = alive ? l : 0.f;
            last_row = row;
            if (rows.rank == 0 && tid == 0)
                a.stats[row] = alive ? make_float2(m, logsum * kLn2) : make_float2(0.f, 0.f);
        }
        place = next_place;
        alive = next_alive;
    }
    if (!BACKWARD) {
        __syncthreads();
        if (rows.rank == 0 && tid == 0) a.loss[last_row] = row_loss(red_loss[par ^ 1], a.tau);
        if (nc > 1) cg::this_cluster().sync();  // nobody leaves while its pair is read
    }
}

// Loss and gradient in one pass. While a row is read and its sums are formed, the gradient of the
// row before it is computed from the copy in shared memory and written: batch by batch, a place's
// old vector is used up, the new row's vector is sent for, and added kLag batches later. So
// memory and the exponent unit see the same load all the time. a.ring batches of a thread have
// a place; what a longer row has behind them is read last and, a barrier later, read again for its
// gradient first (from L2, in practice).
// Threads resident per SM: 768 in CTAs of up to 256, or one CTA of kStepWide for rows that need the
// whole SM's memory (more threads would not get the registers: 640 threads 504 us, 768 534, 1024
// 646 where 512 took 490, for 4096 rows of 131072 bf16 logits; three CTAs of 256 read most of the row a
// second time from HBM, since 444 such rows do not stay in L2: 614). Vectors of a batch, and how many
// batches later it is added.
constexpr int kStepWide = 512, kStepAhead = 256 * 1024;
constexpr int step_threads(int nt) { return nt == kStepWide ? nt : 768; }
constexpr int step_batch(int nt) { return nt == kStepWide ? 4 : 2; }
constexpr int step_lag(int nt) { return nt == kStepWide ? 2 : 3; }

template <typename T, int NT>
__global__ void __launch_bounds__(NT, step_threads(NT) / NT) distill_step_kernel(const DistillArgs a) {
    constexpr int U = step_batch(NT), kLag = step_lag(NT);
    using R = Rows<T, NT, U>;
    using P = typename R::P;
    constexpr int W = R::W;
    extern __shared__ __align__(16) uint4 dyn[];
    __shared__ float2 red_row[2][W], red_slots[2][W], shared_ms[2], row_stats[2];
    __shared__ float red_loss[2][W];
    pdl_wait();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int nc = 1 << a.log_cluster, ring = a.ring;
    const R rows = {a, static_cast<int>(cg::this_cluster().block_rank()), nc, (a.K + 3) & ~3,
                    dyn + tid, reinterpret_cast<int *>(dyn + ring * R::STEP), kLog2e / a.tau};
    const float c = rows.c;

    // `row` is being read, `old_row` gets its gradient
    const int stride = gridDim.x >> a.log_cluster;
    int row = blockIdx.x >> a.log_cluster, old_row = -1, par = 0, place = 0;
    bool alive, old_alive = false;
    {
        int id = -1;
        float x = -INFINITY;
        if (tid < a.K) rows.slot_of(row, tid, id, x);
        alive = __syncthreads_or(rows.list_slots(row, 0, id, x));
    }
    while (row < a.n || old_row >= 0) {
        const bool has_row = row < a.n;
        const int next_row = row + stride;
        const bool has_next = next_row < a.n;
        int next_id = -1;
        float next_x = -INFINITY;
        if (has_next && tid < a.K) rows.slot_of(next_row, tid, next_id, next_x);
        Running r = {-INFINITY, {make_float2(0.f, 0.f), make_float2(0.f, 0.f)}};
        {
            const typename R::Share cur = rows.share_of(has_row ? row : old_row);
            const typename R::Share old = rows.share_of(old_row >= 0 ? old_row : row);
            const int nb = alive ? cur.nb : 0, old_nb = old_alive ? old.nb : 0;
            const float2 st = row_stats[par ^ 1];
            const Gradient<T, NT, U> grad(rows, old_row >= 0 ? old_row : row, st.x, st.y);
            const bool vec = grad.aligned(old);
            if (alive) rows.add_ends(cur, r);
            if (old_alive)
                grad.ends(rows, old);
            else if (old_row >= 0)
                grad.zeros(rows, old);
            // what has no place, of the old row: read last before, so L2 still has it
            rows.walk(old, ring, old_nb, [&](int b, P(&v)[U]) { grad.batch(rows, old, b, vec, v); });
            const int kept = min(nb, ring), old_kept = min(old_nb, ring);
            const int steps = max(old_kept, nb ? kept + kLag : 0);
            const T *p = rows.behind_first(cur) - R::STEP * R::VEC;  // batch b, b > 0
            uint4 *slot = rows.mine;
            for (int b = 0; b < steps; ++b, p += R::STEP * R::VEC, slot += R::STEP) {
                P v[U];
                if (b >= kLag && b - kLag < kept) {
                    cp_async_wait<kLag - 1>();
                    R::take(slot - kLag * R::STEP, v);
                    if (b == kLag) rows.fill(cur, v);
                    rows.add(r, v);
                }
                if (b < old_kept) {
                    R::take(slot, v);
                    grad.batch(rows, old, b, vec, v);
                }
                if (b < kept) {
                    if (b == 0)
                        rows.fetch_first(cur, slot);
                    else
                        R::fetch(p, slot);
                }
                cp_async_commit();
            }
            rows.walk(cur, ring, nb, [&](int, P(&v)[U]) { rows.add(r, v); });
        }

        if (has_next && tid == 0) {
            // the next row, or what kStepAhead holds of it, on its way to L2 while this one is brought
            // to its end, whether or not it turns out to have a slot (sent for at the start of the row
            // it pushes out what is still to be read: 571 us instead of 469)
            const typename R::Share next = rows.share_of(next_row);
            const int bytes = min(next.n, kStepAhead / 16) * 16;
            if (bytes)
                asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(next.zv), "r"(bytes) : "memory");
        }
        // the next row's slots and their logits, read before anything of that row is replaced
        const int next_place = (place + 1) % kPlaces, old_place = (place + kPlaces - 1) % kPlaces;
        bool live = false;
        if (has_next) live = rows.list_slots(next_row, next_place, next_id, next_x);
        MaxSum t = {-INFINITY, 0.f}, q = t;
        if (has_row) {
            t = join_lanes<32>(rows.teacher(place), c);
            q = join_lanes<32>(r.sum(), c);
        }
        if (lane == 0) {
            red_row[par][warp] = make_float2(q.m, q.s);
            red_slots[par][warp] = make_float2(t.m, t.s);
        }
        const bool next_alive = __syncthreads_or(live);
        // the old row: the columns with a slot, and the loss, its parts complete since this barrier
        if (old_row >= 0) {
            if (old_alive) {
                const float2 st = row_stats[par ^ 1];
                Gradient<T, NT, U>(rows, old_row, st.x, st.y).columns(rows, rows.share_of(old_row), old_place);
            }
            if (rows.rank == 0 && tid == 0) a.loss[old_row] = row_loss(red_loss[par ^ 1], a.tau);
        }
        if (has_row) {
            t = join_warps(red_slots[par], c);
            q = join_warps(red_row[par], c);
            if (nc > 1) q = join_cluster(q, &shared_ms[par], nc, c);
            float m;
            const float logsum = log_of(q, m);
            const float l = warp_sum(rows.finish_slots(place, t, m, logsum));
            if (lane == 0) red_loss[par][warp] = alive ? l : 0.f;
            if (tid == 0) row_stats[par] = make_float2(m, logsum);
        }
        __syncthreads();  // the statistics
        old_row = has_row ? row : -1, old_alive = alive;
        row = next_row, alive = next_alive, place = next_place;
        par ^= 1;
    }
    if (nc > 1) cg::this_cluster().sync();  // nobody leaves while its pair is read
}

size_t lists_bytes(int K) { return size_t(kPlaces) * 3 * 4 * ((K + 3) & ~3); }

template <typename Kernel>
cudaError_t launch_rows(Kernel kernel, const DistillArgs &a, int nt, int threads, bool even, size_t smem,
                        int num_sms, cudaStream_t st) {
    int per_sm = threads / nt;
    const int by_smem = static_cast<int>(size_t(226) * 1024 / (smem + 2048));
    if (by_smem < per_sm) per_sm = by_smem < 1 ? 1 : by_smem;
    // at a time; `even`: as many as leave every CTA the same number of them (the loss of 4096 rows:
    // 52 us instead of 55; loss and gradient in one pass lose by it, 132 instead of 125)
    int rows = (per_sm * num_sms) >> a.log_cluster;
    if (rows > a.n) rows = a.n;
    if (even) rows = (a.n + (a.n + rows - 1) / rows - 1) / ((a.n + rows - 1) / rows);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(rows) << a.log_cluster);
    cfg.blockDim = dim3(nt);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 1u << a.log_cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.log_cluster ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

// Shared memory for a.ring batches of loss and gradient in one pass: an even share of an SM's.
constexpr int kStepSmem = 200 * 1024, kSmemMost = 224 * 1024;  // (227 KB less the static part)

// Threads per SM of the gradient's pass. Many long rows: half of what fits, which leaves DRAM longer
// runs (4096 rows of 32768 bf16 logits: 98 us instead of 105; of 16384: 52 either way. Shorter or
// fewer rows want all: 25 instead of 32 for 4096 rows of 8192, 40 instead of 42 for 1000 of 50001,
// 37 instead of 39 for 1500 of 32768; the loss alone of 4096 rows of 32768 takes 59 instead of
// 52 that way).
int gradient_threads(const DistillArgs &a, int size, int num_sms) {
    return a.n >= 16 * num_sms && static_cast<long long>(a.V) * size >= 32768 ? 512 : 1024;
}

template <typename T, int MODE, int NT>
cudaError_t launch(DistillArgs a, int num_sms, cudaStream_t st) {
    constexpr int batch = NT * 16 * (MODE == kStep ? step_batch(NT) : kPassBatch);
    if constexpr (MODE == kStep) {
        const int nv = a.V / (16 / static_cast<int>(sizeof(T)));
        const int per = (nv + (1 << a.log_cluster) - 1) >> a.log_cluster;
        const int share = kStepSmem / (step_threads(NT) / NT);
        const int left = kSmemMost - static_cast<int>(lists_bytes(a.K));
        const int nb = static_cast<int>((per * 16LL + batch - 1) / batch);
        const int most = (share < left ? share : left) / batch;
        a.ring = nb < 1 ? 1 : nb < most ? nb : most;
        return launch_rows(distill_step_kernel<T, NT>, a, NT, step_threads(NT), false,
                           size_t(a.ring) * batch + lists_bytes(a.K), num_sms, st);
    } else {
        return launch_rows(distill_kernel<T, MODE == kBackward, NT>, a, NT,
                           MODE == kBackward ? gradient_threads(a, static_cast<int>(sizeof(T)), num_sms) : 1024, true,
                           size_t(kRing) * batch + lists_bytes(a.K), num_sms, st);
    }
}

template <typename T, int MODE>
cudaError_t launch_nt(const DistillArgs &a, int nt, int num_sms, cudaStream_t st) {
    if constexpr (MODE == kStep)
        if (nt == kStepWide) return launch<T, MODE, kStepWide>(a, num_sms, st);
    return nt == 64    ? launch<T, MODE, 64>(a, num_sms, st)
           : nt == 128 ? launch<T, MODE, 128>(a, num_sms, st)
                       : launch<T, MODE, 256>(a, num_sms, st);
}

template <typename T>
cudaError_t launch_mode(const DistillArgs &a, int mode, int nt, int num_sms, cudaStream_t st) {
    switch (mode) {
        case kForward: return launch_nt<T, kForward>(a, nt, num_sms, st);
        case kBackward: return launch_nt<T, kBackward>(a, nt, num_sms, st);
        default: return launch_nt<T, kStep>(a, nt, num_sms, st);
    }
}

template <typename T, int NT>
cudaError_t configure() {
    constexpr auto attr = cudaFuncAttributeMaxDynamicSharedMemorySize;
    const int lists = static_cast<int>(lists_bytes(RSA_DISTILL_MAX_K));
    const int pass = kRing * NT * kPassBatch * 16 + lists, step = kStepSmem / (step_threads(NT) / NT) + lists;
    cudaError_t e = cudaSuccess;
    e = cudaFuncSetAttribute(distill_kernel<T, false, NT>, attr, pass);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(distill_kernel<T, true, NT>, attr, pass);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(distill_step_kernel<T, NT>, attr, step);
    if (NT == 256 && e == cudaSuccess)
        e = cudaFuncSetAttribute(distill_step_kernel<T, kStepWide>, attr,
                                 kStepSmem + lists < kSmemMost ? kStepSmem + lists : kSmemMost);
    return e;
}

}  // namespace

// Threads and CTAs per row. Small CTAs wait less for one another (64 threads: 51 us, 128: 57, 256:
// 72 for the loss of 4096 rows of 32768 bf16 logits), but rows times threads have to fill the GPU,
// and a thread should have four vectors. With loss and gradient in one pass a row wants as much
// shared memory as it has bytes, and so as many threads as go with it.
cudaError_t launch_distill(DistillArgs a, int mode, int bf16, int num_sms, cudaStream_t st) {
    const int nv = a.V / (bf16 ? 8 : 4);
    const long long fill = (mode == kStep ? 600LL : 800LL) * num_sms;  // most of the resident threads
    a.log_cluster = 0;
    int nt = 64;
    if (mode == kStep) {
        while (a.log_cluster < 3 && (a.n * 2LL << a.log_cluster) <= 2 * num_sms &&
               (nv >> a.log_cluster) > 4 * 256)
            ++a.log_cluster;
        while (nt < kStepWide && (nv >> a.log_cluster) * 16LL > kStepSmem / (step_threads(nt) / nt))
            nt = nt == 256 ? kStepWide : 2 * nt;
    }
    while (nt < 256 && a.n * static_cast<long long>(nt << a.log_cluster) < fill &&
           (nv >> a.log_cluster) > 4 * nt)
        nt *= 2;
    while (mode != kStep && a.log_cluster < 3 &&
           a.n * static_cast<long long>(nt << a.log_cluster) < fill && (nv >> a.log_cluster) > 4 * nt)
        ++a.log_cluster;
    return bf16 ? launch_mode<__nv_bfloat16>(a, mode, nt, num_sms, st)
                : launch_mode<float>(a, mode, nt, num_sms, st);
}

cudaError_t distill_kernels_configure() {
    cudaError_t e;
    if ((e = configure<__nv_bfloat16, 64>()) != cudaSuccess ||
        (e = configure<__nv_bfloat16, 128>()) != cudaSuccess ||
        (e = configure<__nv_bfloat16, 256>()) != cudaSuccess ||
        (e = configure<float, 64>()) != cudaSuccess || (e = configure<float, 128>()) != cudaSuccess)
        return e;
    return configure<float, 256>();
}

}  // namespace rsa
