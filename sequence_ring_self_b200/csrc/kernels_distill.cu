// kernels_distill.cu -- distillation from a teacher's top logits: loss, gradient, or both in
// one pass (rsa_distill*, rsa_rows.h).
//
//   p = softmax(teacher / tau) over a row's live slots,  q = softmax(z / tau) over its V logits
//   loss = tau^2 sum_j p_j (ln p_j - ln q_{index_j}),    dz = dloss tau (q - p)
//
// Bound by memory (a row is V elements read, and V written by the gradient), with the exponent
// unit close behind: one exponential per element and pass. A row belongs to one CTA, or to a
// cluster that shares its columns when there are few rows. Every thread keeps a running maximum
// and sum of exponentials of the 16-byte vectors it reads, the CTA joins them by shuffles and
// the cluster through distributed shared memory, always in the same order. The teacher's slots
// lie in shared memory; the gradient is streamed as dloss tau q, and the few columns with a slot
// are written once more afterwards, from logits read before the stream began (which lets the
// gradient replace the logits in place).
#include <cooperative_groups.h>
#include <type_traits>

#include "rows_common.cuh"

namespace rsa {
namespace {

using namespace rows;
namespace cg = cooperative_groups;

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kUnroll = 4;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// 2^x by the hardware's approximation (about 2 units in the last place). Results below the
// smallest normal number flush to zero: a probability below 2^-126 adds nothing to a sum that
// is at least 1, and rounds to no bf16 or fp32 gradient that matters next to it.
__device__ __forceinline__ float exp2_ftz(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Running maximum m and s = sum 2^((z - m) c). Differences are taken before the scaling, so a
// logit of the type's lowest value cannot overflow against another of the same.
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

template <int N>
__device__ __forceinline__ void add(MaxSum &r, const float (&f)[N], float c) {
    float m = f[0];
#pragma unroll
    for (int e = 1; e < N; ++e) m = fmaxf(m, f[e]);
    if (m > r.m) {
        r.s *= exp2_ftz((r.m - m) * c);
        r.m = m;
    }
    const float ref = r.m == -INFINITY ? 0.f : r.m;
#pragma unroll
    for (int e = 0; e < N; ++e) r.s += exp2_ftz((f[e] - ref) * c);
}

__device__ __forceinline__ float block_sum(float x, float *tmp) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) tmp[threadIdx.x >> 5] = x;
    __syncthreads();
    x = tmp[threadIdx.x & (kWarps - 1)];
#pragma unroll
    for (int o = kWarps / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

__device__ __forceinline__ MaxSum block_max_sum(MaxSum r, float c, float2 *tmp) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        r = join(r, {__shfl_xor_sync(0xffffffffu, r.m, o), __shfl_xor_sync(0xffffffffu, r.s, o)}, c);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) tmp[threadIdx.x >> 5] = make_float2(r.m, r.s);
    __syncthreads();
    const float2 v = tmp[threadIdx.x & (kWarps - 1)];
    r = {v.x, v.y};
#pragma unroll
    for (int o = kWarps / 2; o > 0; o >>= 1)
        r = join(r, {__shfl_xor_sync(0xffffffffu, r.m, o), __shfl_xor_sync(0xffffffffu, r.s, o)}, c);
    return r;
}

enum { kForward, kBackward, kStep };

template <typename T, int MODE>
__global__ void __launch_bounds__(kThreads) distill_kernel(const DistillArgs a) {
    constexpr int VEC = 16 / sizeof(T);
    using P = Pack<T, VEC>;
    extern __shared__ float dyn[];  // per slot: index, teacher logit then probability, logit
    __shared__ float red[kWarps];
    __shared__ float2 red2[kWarps];
    __shared__ float2 shared_ms;
    pdl_wait();
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = static_cast<int>(cluster.block_rank()), nc = a.cluster;
    const int tid = threadIdx.x, K = a.K, V = a.V;
    const long long row = blockIdx.x / static_cast<unsigned>(nc);
    const T *z = static_cast<const T *>(a.z) + row * a.ld;
    T *dz = MODE == kForward ? nullptr : static_cast<T *>(a.dz) + row * a.ld_d;
    int *slot = reinterpret_cast<int *>(dyn);
    float *prob = dyn + K, *zs = dyn + 2 * K;
    const float c = kLog2e / a.tau;

    // this CTA's columns: `head` single elements up to the first 16-byte boundary (rank 0),
    // then vectors [v0, v1), then single elements behind the last vector (the last rank)
    const int mis = static_cast<int>(reinterpret_cast<uintptr_t>(z) / sizeof(T)) & (VEC - 1);
    const int head = min(V, mis ? VEC - mis : 0), nv = (V - head) / VEC, tail = head + nv * VEC;
    const int per = (nv + nc - 1) / nc;
    const int v0 = min(nv, rank * per), v1 = min(nv, v0 + per);
    const int lo = rank ? head + v0 * VEC : 0, hi = rank == nc - 1 ? V : head + v1 * VEC;

    // the teacher's slots
    MaxSum t = {-INFINITY, 0.f};
    for (int j = tid; j < K; j += kThreads) {
        const long long id = index_at(a.index, a.index64, row * K + j);
        const long long at = row * K + j;
        const float x = a.teacher_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(a.teacher)[at])
                                       : static_cast<const float *>(a.teacher)[at];
        const bool live = id >= 0 && id < V && x != -INFINITY;
        slot[j] = live ? static_cast<int>(id) : -1;
        prob[j] = x;
        if (live) {
            zs[j] = static_cast<float>(z[id]);
            t = join(t, {x, 1.f}, c);
        }
    }
    const bool any = __syncthreads_or(t.s != 0.f);
    if (!any) {  // the same answer in every CTA of the row
        if (MODE != kForward)
            for (int i = lo + tid; i < hi; i += kThreads) dz[i] = T(0.f);
        if (rank == 0 && tid == 0) {
            if (MODE != kBackward) a.loss[row] = 0.f;
            if (MODE == kForward) a.stats[row] = make_float2(0.f, 0.f);
        }
        return;
    }
    t = block_max_sum(t, c, red2);
    const float tl2 = log2f(t.s);

    // maximum and sum of the row's exponentials
    float m, logsum;  // max z, log2 of the sum
    if (MODE == kBackward) {
        const float2 st = static_cast<const float2 *>(a.stats)[row];
        m = st.x, logsum = st.y * kLog2e;
    } else {
        MaxSum r = {-INFINITY, 0.f};
        if (rank == 0 && tid < head) {
            const float f[1] = {static_cast<float>(z[tid])};
            add<1>(r, f, c);
        }
        if (rank == nc - 1 && tid < V - tail) {
            const float f[1] = {static_cast<float>(z[tail + tid])};
            add<1>(r, f, c);
        }
        for (int i = v0 + tid; i < v1; i += kThreads * kUnroll) {
            P v[kUnroll];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u)
                if (i + u * kThreads < v1) v[u] = P::load(z + head + (i + u * kThreads) * static_cast<long long>(VEC));
#pragma unroll
            for (int u = 0; u < kUnroll; ++u)
                if (i + u * kThreads < v1) {
                    float f[VEC];
                    v[u].to(f);
                    add<VEC>(r, f, c);
                }
        }
        r = block_max_sum(r, c, red2);
        if (nc > 1) {
            if (tid == 0) shared_ms = make_float2(r.m, r.s);
            cluster.sync();
            r = {-INFINITY, 0.f};
            for (int i = 0; i < nc; ++i) {
                const float2 v = *cluster.map_shared_rank(&shared_ms, i);
                r = join(r, {v.x, v.y}, c);
            }
            cluster.sync();  // nobody leaves while its pair is read
        }
        m = r.m, logsum = log2f(r.s);
        if (r.s != r.s && m != INFINITY) m = r.s;  // a NaN in the row
        if (m == -INFINITY) logsum = NAN;          // no logit at all: no softmax
    }

    // probabilities and, on one CTA, the loss
    float l = 0.f;
    for (int j = tid; j < K; j += kThreads) {
        const float lp = (prob[j] - t.m) * c - tl2;  // log2 p
        const float p = slot[j] >= 0 ? exp2_ftz(lp) : 0.f;
        if (MODE != kBackward && p != 0.f) l += p * (lp - ((zs[j] - m) * c - logsum));
        prob[j] = p;
    }
    if (MODE != kBackward && rank == 0) {
        l = block_sum(l, red);
        if (tid == 0) {
            a.loss[row] = a.tau * a.tau * kLn2 * l;
            if (MODE == kForward) a.stats[row] = make_float2(m, logsum * kLn2);
        }
    }
    if (MODE == kForward) return;

    // the gradient: g q everywhere, then g (q - p) where a slot points
    const float g = a.dloss[row * a.dloss_stride] * a.tau;
    auto grad = [&](float x, float p) { return g * (exp2_ftz((x - m) * c - logsum) - p); };
    if (rank == 0 && tid < head) dz[tid] = T(grad(static_cast<float>(z[tid]), 0.f));
    if (rank == nc - 1 && tid < V - tail) dz[tail + tid] = T(grad(static_cast<float>(z[tail + tid]), 0.f));
    const bool aligned = ((reinterpret_cast<uintptr_t>(z) ^ reinterpret_cast<uintptr_t>(dz)) & 15u) == 0;
    for (int i = v0 + tid; i < v1; i += kThreads * kUnroll) {
        P v[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            if (i + u * kThreads < v1) v[u] = P::load(z + head + (i + u * kThreads) * static_cast<long long>(VEC));
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            if (i + u * kThreads < v1) {
                float f[VEC];
                v[u].to(f);
#pragma unroll
                for (int e = 0; e < VEC; ++e) f[e] = grad(f[e], 0.f);
                T *to = dz + head + (i + u * kThreads) * static_cast<long long>(VEC);
                if (aligned) {
                    P::from(f).store(to);
                } else {
#pragma unroll
                    for (int e = 0; e < VEC; ++e) to[e] = T(f[e]);
                }
            }
    }
    __syncthreads();  // the streamed values are written, the probabilities are in place
    for (int j = tid; j < K; j += kThreads) {
        const int id = slot[j];
        if (id < lo || id >= hi) continue;
        float p = 0.f;  // slots with the same index add up
        for (int i = 0; i < K; ++i) p += slot[i] == id ? prob[i] : 0.f;
        dz[id] = T(grad(zs[j], p));
    }
}

template <typename T, int MODE>
cudaError_t launch(const DistillArgs &a, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.n) * a.cluster);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = size_t(12) * a.K;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = a.cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, distill_kernel<T, MODE>, a);
}

template <typename T>
cudaError_t launch_mode(const DistillArgs &a, int mode, cudaStream_t st) {
    switch (mode) {
        case kForward: return launch<T, kForward>(a, st);
        case kBackward: return launch<T, kBackward>(a, st);
        default: return launch<T, kStep>(a, st);
    }
}

}  // namespace

// CTAs per row: more only while the rows alone leave SMs idle and each CTA keeps a vector or
// two for every thread.
cudaError_t launch_distill(DistillArgs a, int mode, int bf16, int num_sms, cudaStream_t st) {
    const int vec = bf16 ? 8 : 4;
    a.cluster = 1;
    while (a.cluster < 8 && static_cast<long long>(a.n) * a.cluster < 2 * num_sms &&
           a.V / (vec * kThreads * a.cluster) >= 2)
        a.cluster *= 2;
    return bf16 ? launch_mode<__nv_bfloat16>(a, mode, st) : launch_mode<float>(a, mode, st);
}

}  // namespace rsa
