// kernels_embed.cu -- embedding lookup and the gradient of its table (rsa_embed, rsa_rows.h).
//
// Lookup: bound by memory, out[t] = scale * table[ids[t]] moved in 16-byte vectors, four per
// thread in flight.
//
// Gradient: dtable[v] = scale * sum of the rows of dout whose id is v. The tokens are sorted by
// id with a stable radix sort, the sorted list is cut into pieces of S tokens, and every piece
// adds up its rows in order, fp32 in registers, one 16-byte column per thread. An id whose
// tokens lie inside one piece is written at once; one that spans pieces leaves a partial row in
// each, and a last kernel adds those in order. So each dout row is read once, a token that
// fills half the batch is shared by many blocks, and the order of every sum is fixed.
#include <cooperative_groups.h>
#include <type_traits>

#include "rows_common.cuh"

namespace rsa {
namespace {

using namespace rows;
namespace cg = cooperative_groups;

// ------------------------------------------------------------------ lookup

constexpr int kLookupThreads = 256, kLookupUnits = 4;

// A unit is one access of N elements; a warp serves 128 consecutive units of the rows' list.
template <typename T, int N>
__global__ void __launch_bounds__(kLookupThreads) embed_kernel(const EmbedArgs a) {
    using P = Pack<T, N>;
    pdl_wait();
    const unsigned nu = a.D / N;  // units per row
    const unsigned long long total = static_cast<unsigned long long>(a.n) * nu;
    const unsigned long long first =
        (blockIdx.x * static_cast<unsigned long long>(kLookupThreads / 32) + (threadIdx.x >> 5)) *
        (32 * kLookupUnits);
    if (first >= total) return;
    const unsigned row0 = static_cast<unsigned>(first / nu);
    const unsigned rem0 = static_cast<unsigned>(first - static_cast<unsigned long long>(row0) * nu);
    P v[kLookupUnits];
    long long to[kLookupUnits];
#pragma unroll
    for (int u = 0; u < kLookupUnits; ++u) {
        const unsigned off = rem0 + u * 32 + (threadIdx.x & 31);
        const unsigned r = off / nu, col = (off - r * nu) * N, row = row0 + r;
        const bool on = first + u * 32 + (threadIdx.x & 31) < total;
        to[u] = on ? row * a.ld_out + col : -1;
        const long long id = on ? index_at(a.ids, a.ids64, row) : -1;
        v[u] = id >= 0 && id < a.V
                   ? P::load(static_cast<const T *>(a.table) + id * a.ld_table + col)
                   : P::zero();
    }
#pragma unroll
    for (int u = 0; u < kLookupUnits; ++u) {
        if (to[u] < 0) continue;
        float f[N];
        v[u].to(f);
#pragma unroll
        for (int e = 0; e < N; ++e) f[e] *= a.scale;
        P::from(f).store(static_cast<T *>(a.out) + to[u]);
    }
}

// ------------------------------------------------------------------ sort by id

constexpr int kSortThreads = 1024, kSortWarps = kSortThreads / 32, kSortCluster = 8;
constexpr int kSortMaxBits = 10;  // digits: 32 warps x 1024 counters = 128 KB

// Stable LSD radix sort of the n (id, token) pairs by one cluster, any n: each warp of the
// cluster owns a contiguous run of tokens; per pass it counts its digits (32 tokens at a time,
// equal digits found by a match over the warp), the cluster adds the counts up over warps,
// CTAs and digits through distributed shared memory, and the warps place their tokens in
// order. The lists lie in global memory (in practice in L2); the cluster's barriers order the
// passes. Ids outside [0, V) become V and sort last. The other clusters of the grid meanwhile
// fill the table's gradient with zeros.
template <typename TO, int N>
__global__ void __cluster_dims__(kSortCluster, 1, 1) __launch_bounds__(kSortThreads, 1)
    embed_sort_kernel(const EmbedArgs a) {
    pdl_wait();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (blockIdx.x >= kSortCluster) {
        const unsigned nu = a.D / N;
        const unsigned stride = (gridDim.x - kSortCluster) * kSortWarps;
        for (unsigned r = (blockIdx.x - kSortCluster) * kSortWarps + warp;
             r < static_cast<unsigned>(a.V); r += stride) {
            TO *row = static_cast<TO *>(a.dtable) + r * a.ld_dtable;
            for (unsigned c = lane; c < nu; c += 32) Pack<TO, N>::zero().store(row + c * N);
        }
        return;
    }
    extern __shared__ uint32_t cnt[];  // [warps][digits], then total[digits], base[digits]
    __shared__ uint32_t wsum[kSortWarps];
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = static_cast<int>(cluster.block_rank());
    const int nd = 1 << a.bits;
    uint32_t *mine = cnt + warp * nd, *total = cnt + kSortWarps * nd, *base = total + nd;
    if (rank == 0 && tid == 0) *a.count = 0;
    // per-warp runs of whole 32-token rounds
    const unsigned n = a.n, all = kSortCluster * kSortThreads;
    const unsigned run = (n + all - 1) / all * 32;
    const unsigned long long s0 = static_cast<unsigned long long>(rank * kSortWarps + warp) * run;
    const unsigned start = s0 < n ? static_cast<unsigned>(s0) : n;
    const unsigned end = n - start < run ? n : start + run;
    const uint32_t below = (1u << lane) - 1u;
    for (int pass = 0; pass < a.passes; ++pass) {
        // pass 0 reads the ids; the last pass writes to (key[0], idx[0])
        const int to = (a.passes - 1 - pass) & 1;
        const uint32_t *key_in = a.key[to ^ 1], *idx_in = a.idx[to ^ 1];
        uint32_t *key_out = a.key[to], *idx_out = a.idx[to];
        const int shift = pass * a.bits;
        auto key_of = [&](unsigned t) -> uint32_t {
            if (pass) return key_in[t];
            const long long id = index_at(a.ids, a.ids64, t);
            return id >= 0 && id < a.V ? static_cast<uint32_t>(id) : static_cast<uint32_t>(a.V);
        };
        for (int i = tid; i < kSortWarps * nd; i += kSortThreads) cnt[i] = 0;
        __syncthreads();
        for (unsigned t0 = start; t0 < end; t0 += 32) {
            const bool on = t0 + lane < end;
            const uint32_t dig = on ? (key_of(t0 + lane) >> shift) & (nd - 1) : ~0u;
            const uint32_t peers = __match_any_sync(0xffffffffu, dig);
            if (on && !(peers & below)) mine[dig] += __popc(peers);
            __syncwarp();
        }
        __syncthreads();
        if (tid < nd) {  // counts -> first place of each warp inside the CTA's share of a digit
            uint32_t s = 0;
#pragma unroll 8
            for (int w = 0; w < kSortWarps; ++w) {
                const uint32_t c = cnt[w * nd + tid];
                cnt[w * nd + tid] = s;
                s += c;
            }
            total[tid] = s;
        }
        cluster.sync();
        uint32_t before = 0, sum = 0;
        if (tid < nd) {
#pragma unroll
            for (int c = 0; c < kSortCluster; ++c) {
                const uint32_t v = cluster.map_shared_rank(total, c)[tid];
                before += c < rank ? v : 0;
                sum += v;
            }
        }
        // exclusive sum over the digits, one per thread
        uint32_t inc = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t v = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += v;
        }
        if (lane == 31) wsum[warp] = inc;
        __syncthreads();
        if (warp == 0) {
            uint32_t v = wsum[lane], w = v;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t x = __shfl_up_sync(0xffffffffu, w, o);
                if (lane >= o) w += x;
            }
            wsum[lane] = w - v;
        }
        __syncthreads();
        if (tid < nd) base[tid] = wsum[warp] + inc - sum + before;
        __syncthreads();
        for (unsigned t0 = start; t0 < end; t0 += 32) {
            const unsigned t = t0 + lane;
            const bool on = t < end;
            const uint32_t key = on ? key_of(t) : 0;
            const uint32_t dig = on ? (key >> shift) & (nd - 1) : ~0u;
            const uint32_t peers = __match_any_sync(0xffffffffu, dig);
            if (on) {
                const uint32_t at = base[dig] + mine[dig] + __popc(peers & below);
                key_out[at] = key;
                idx_out[at] = pass ? idx_in[t] : t;
            }
            __syncwarp();
            if (on && !(peers & below)) mine[dig] += __popc(peers);
            __syncwarp();
        }
        // this pass's lists are whole, and nobody reads this CTA's totals any more
        cluster.sync();
    }
}

// ------------------------------------------------------------------ sums of the sorted rows

constexpr int kGradUnroll = 8;

// N sums of row `key` of the table's gradient, from column col: scaled, added to what is there
// when asked to, rounded once.
template <typename TO, int N>
__device__ __forceinline__ void finish(const EmbedArgs &a, uint32_t key, int col, const float (&s)[N]) {
    constexpr int W = N == 1 ? 1 : 16 / sizeof(TO);
    TO *p = static_cast<TO *>(a.dtable) + key * a.ld_dtable + col;
#pragma unroll
    for (int c = 0; c < N; c += W) {
        float f[W];
        if (a.accumulate) {
            Pack<TO, W>::load(p + c).to(f);
#pragma unroll
            for (int e = 0; e < W; ++e) f[e] = fmaf(s[c + e], a.scale, f[e]);
        } else {
#pragma unroll
            for (int e = 0; e < W; ++e) f[e] = s[c + e] * a.scale;
        }
        Pack<TO, W>::from(f).store(p + c);
    }
}

// A partial row: fp32, 16-byte aligned for N > 1.
template <int N>
__device__ __forceinline__ void store_part(float *p, const float (&s)[N]) {
    if constexpr (N == 1) {
        p[0] = s[0];
    } else {
#pragma unroll
        for (int c = 0; c < N; c += 4)
            *reinterpret_cast<float4 *>(p + c) = make_float4(s[c], s[c + 1], s[c + 2], s[c + 3]);
    }
}

// Block (x: columns of N elements, y: pieces). A piece's first id may have begun before it
// (partial row 0) and its last may go on behind it (partial row 1, when it began inside).
template <typename T, typename TO, int N>
__global__ void __launch_bounds__(256) embed_grad_kernel(const EmbedArgs a) {
    using P = Pack<T, N>;
    pdl_wait();
    const unsigned piece = blockIdx.x * blockDim.y + threadIdx.y;
    const int unit = blockIdx.y * blockDim.x + threadIdx.x;
    if (piece >= static_cast<unsigned>(a.npieces) || unit * N >= a.D) return;
    const int col = unit * N;
    const uint32_t *key = a.key[0], *idx = a.idx[0];
    const unsigned begin = piece * static_cast<unsigned>(a.S), n = a.n;
    const unsigned end = n - begin < static_cast<unsigned>(a.S) ? n : begin + a.S;
    const T *dout = static_cast<const T *>(a.dout) + col;
    float *part = a.part + static_cast<size_t>(piece) * 2 * a.Dp + col;
    const uint32_t V = a.V;

    float s[N];
#pragma unroll
    for (int e = 0; e < N; ++e) s[e] = 0.f;
    uint32_t cur = key[begin];
    bool began = begin == 0 || key[begin - 1] != cur;  // cur's first token lies in this piece
    for (unsigned i0 = begin; i0 < end; i0 += kGradUnroll) {
        uint32_t k[kGradUnroll];
        P v[kGradUnroll];
#pragma unroll
        for (int u = 0; u < kGradUnroll; ++u) {
            const unsigned i = i0 + u;
            k[u] = i < end ? key[i] : V;
            v[u] = k[u] < V ? P::load(dout + idx[i] * a.ld_dout) : P::zero();
        }
#pragma unroll
        for (int u = 0; u < kGradUnroll; ++u) {
            if (i0 + u < end && k[u] != cur) {
                if (began) {
                    finish<TO, N>(a, cur, col, s);
                } else {
                    store_part<N>(part, s);
                }
                began = true;
                cur = k[u];
#pragma unroll
                for (int e = 0; e < N; ++e) s[e] = 0.f;
            }
            float f[N];
            v[u].to(f);
#pragma unroll
            for (int e = 0; e < N; ++e) s[e] += f[e];
        }
    }
    if (cur >= V) return;  // ids outside the table come last
    const bool more = end < n && key[end] == cur;
    if (began && !more) {
        finish<TO, N>(a, cur, col, s);
    } else {
        store_part<N>(part + (began ? a.Dp : 0), s);
        if (began && unit == 0) a.list[atomicAdd(a.count, 1u)] = piece;
    }
}

// The ids that span pieces: for each listed piece p, its partial row 1 plus the rows 0 of the
// pieces that follow while the id goes on. Block: 32 x 4 columns, 8 slices of the pieces.
template <typename TO>
__global__ void __launch_bounds__(256) embed_join_kernel(const EmbedArgs a) {
    __shared__ float4 sums[8][32];
    pdl_wait();
    const int lane = threadIdx.x & 31, y = threadIdx.x >> 5;
    const int col = (blockIdx.y * 32 + lane) * 4;
    const uint32_t count = *a.count;
    for (uint32_t i = blockIdx.x; i < count; i += gridDim.x) {
        const unsigned p = a.list[i];
        const uint32_t id = a.key[0][p * static_cast<unsigned>(a.S)  + a.S - 1];
        // the pieces p + 1 .. p + m hold the rest: piece q has some of it when its first is id
        unsigned m = 0;
        for (;;) {
            const unsigned q = p + 1 + m + lane;
            const bool has = q < static_cast<unsigned>(a.npieces) &&
                             a.key[0][q * static_cast<unsigned>(a.S)] == id;
            const uint32_t not_in = ~__ballot_sync(0xffffffffu, has);
            if (not_in) {
                m += __ffs(not_in) - 1;
                break;
            }
            m += 32;
        }
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        if (col < a.Dp) {
            // rows 0 .. m: row 0 is piece p's partial row 1, row j > 0 piece (p + j)'s row 0
            const unsigned per = (m + 8) / 8, j1 = min((y + 1) * per, m + 1);
#pragma unroll 4
            for (unsigned j = y * per; j < j1; ++j) {
                const float4 v = *reinterpret_cast<const float4 *>(
                    a.part + (static_cast<size_t>(p + j) * 2 + (j == 0)) * a.Dp + col);
                s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
            }
        }
        sums[y][lane] = s;
        __syncthreads();
        if (y == 0) {
#pragma unroll
            for (int w = 1; w < 8; ++w) {
                const float4 v = sums[w][lane];
                s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
            }
            const float f[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float one[1] = {f[e]};
                if (col + e < a.D) finish<TO, 1>(a, id, col + e, one);
            }
        }
        __syncthreads();
    }
}

template <typename T, int N>
cudaError_t launch_lookup(const EmbedArgs &a, cudaStream_t st) {
    const unsigned long long units = static_cast<unsigned long long>(a.n) * (a.D / N);
    const unsigned long long per = kLookupThreads * kLookupUnits;
    return launch_pdl(embed_kernel<T, N>, dim3(static_cast<unsigned>((units + per - 1) / per)),
                      dim3(kLookupThreads), 0, st, a);
}

size_t sort_smem(int bits) { return (size_t(kSortWarps) + 2) * (size_t(4) << bits); }

template <typename T, typename TO, int N>
cudaError_t launch_grad(const EmbedArgs &a, cudaStream_t st) {
    const int units = a.D / N;
    const int tx = units < 256 ? units : 256, ty = 256 / tx;
    return launch_pdl(embed_grad_kernel<T, TO, N>,
                      dim3((a.npieces + ty - 1) / ty, (units + tx - 1) / tx), dim3(tx, ty), 0, st, a);
}

template <typename T, typename TO>
cudaError_t launch_grad_w(const EmbedArgs &a, int vec, cudaStream_t st) {
    return vec ? launch_grad<T, TO, 16 / sizeof(T)>(a, st) : launch_grad<T, TO, 1>(a, st);
}

}  // namespace

cudaError_t launch_embed(const EmbedArgs &a, int bf16, int vec, cudaStream_t st) {
    if (bf16)
        return vec ? launch_lookup<__nv_bfloat16, 8>(a, st) : launch_lookup<__nv_bfloat16, 1>(a, st);
    return vec ? launch_lookup<float, 4>(a, st) : launch_lookup<float, 1>(a, st);
}

// Digits: the fewest passes of at most kSortMaxBits bits over the values 0 .. V.
void embed_sort_plan(EmbedArgs &a) {
    int bits = 1;
    while (bits < 31 && (a.V >> bits)) ++bits;
    a.passes = (bits + kSortMaxBits - 1) / kSortMaxBits;
    a.bits = (bits + a.passes - 1) / a.passes;
}

cudaError_t launch_embed_sort(const EmbedArgs &a, int bf16_out, int vec, int num_sms,
                              cudaStream_t st) {
    const int clusters = a.accumulate ? 1 : num_sms / kSortCluster;
    const dim3 grid((clusters > 2 ? clusters : a.accumulate ? 1 : 2) * kSortCluster);
    const size_t smem = sort_smem(a.bits);
    if (bf16_out)
        return vec ? launch_pdl(embed_sort_kernel<__nv_bfloat16, 8>, grid, dim3(kSortThreads), smem, st, a)
                   : launch_pdl(embed_sort_kernel<__nv_bfloat16, 1>, grid, dim3(kSortThreads), smem, st, a);
    return vec ? launch_pdl(embed_sort_kernel<float, 4>, grid, dim3(kSortThreads), smem, st, a)
               : launch_pdl(embed_sort_kernel<float, 1>, grid, dim3(kSortThreads), smem, st, a);
}

cudaError_t launch_embed_grad(const EmbedArgs &a, int bf16, int bf16_out, int vec, cudaStream_t st) {
    if (!bf16) return launch_grad_w<float, float>(a, vec, st);
    return bf16_out ? launch_grad_w<__nv_bfloat16, __nv_bfloat16>(a, vec, st)
                    : launch_grad_w<__nv_bfloat16, float>(a, vec, st);
}

cudaError_t launch_embed_join(const EmbedArgs &a, int bf16_out, int num_sms, cudaStream_t st) {
    const dim3 grid(a.npieces < 2 * num_sms ? a.npieces : 2 * num_sms, (a.Dp / 4 + 31) / 32);
    return bf16_out ? launch_pdl(embed_join_kernel<__nv_bfloat16>, grid, dim3(256), 0, st, a)
                    : launch_pdl(embed_join_kernel<float>, grid, dim3(256), 0, st, a);
}

cudaError_t embed_kernels_configure() {
    const int smem = static_cast<int>(sort_smem(kSortMaxBits));
    const void *kernels[] = {reinterpret_cast<const void *>(embed_sort_kernel<__nv_bfloat16, 8>),
                             reinterpret_cast<const void *>(embed_sort_kernel<__nv_bfloat16, 1>),
                             reinterpret_cast<const void *>(embed_sort_kernel<float, 4>),
                             reinterpret_cast<const void *>(embed_sort_kernel<float, 1>)};
    for (const void *k : kernels) {
        const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace rsa
