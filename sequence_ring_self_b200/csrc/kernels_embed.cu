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

constexpr int kSortThreads = 512, kSortWarps = kSortThreads / 32;
constexpr int kSortMaxBits = 9;  // digits: one per thread; 16 warps x 512 counters = 32 KB

constexpr int kSortKeep = 4;  // rounds of 32 tokens that a warp loads at once

// Stable LSD radix sort of the n (id, token) pairs by one cluster, any n: each warp of the
// cluster owns a contiguous run of tokens; per pass it counts its digits (32 tokens at a time,
// equal digits found by a ballot per bit; __match_any_sync took twice as long), the cluster adds the counts up over warps,
// CTAs and digits through distributed shared memory, and the warps place their tokens in
// order. The lists lie in global memory (in practice in L2); the cluster's barriers order the
// passes. Ids outside [0, V) become V and sort last. Bound by latency: about five dependent trips
// to L2 or a neighbouring SM per pass (alone: 10.5 us for 8192 tokens, 15 for 16384).
//
// Unless the sums are added to what is there, the grid has more clusters, which meanwhile fill the
// gradient with zeros in accesses of N elements, a row per warp (as a kernel of its own beside
// the sort's this was no use: the cluster waits for SMs without other work).
template <typename TO, int N>
__global__ void __launch_bounds__(kSortThreads, 2) embed_sort_kernel(const EmbedArgs a) {
    pdl_wait();
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = static_cast<int>(cluster.block_rank()), nc = a.sort_ctas;
    if (blockIdx.x >= static_cast<unsigned>(nc)) {
        const unsigned nu = a.D / N, stride = (gridDim.x - nc) * kSortWarps;
        for (unsigned r = (blockIdx.x - nc) * kSortWarps + (threadIdx.x >> 5);
             r < static_cast<unsigned>(a.V); r += stride) {
            TO *row = static_cast<TO *>(a.dtable) + r * a.ld_dtable;
            for (unsigned c = threadIdx.x & 31; c < nu; c += 32) Pack<TO, N>::zero().store(row + c * N);
        }
        return;
    }
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    extern __shared__ uint32_t cnt[];  // [warps][digits], then total[digits], base[digits]
    __shared__ uint32_t wsum[kSortWarps];
    auto sync_all = [&]() {
        if (nc > 1)
            cluster.sync();
        else
            __syncthreads();
    };
    const int nd = 1 << a.bits;
    uint32_t *mine = cnt + warp * nd, *total = cnt + kSortWarps * nd, *base = total + nd;
    if (rank == 0 && tid == 0) *a.count = 0;
    // per-warp runs of whole 32-token rounds
    const unsigned n = a.n, all = nc * kSortThreads;
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
        uint32_t key[kSortKeep], idx[kSortKeep], peers[kSortKeep];
        auto load = [&](unsigned t0) {
#pragma unroll
            for (int k = 0; k < kSortKeep; ++k) {
                const unsigned t = t0 + k * 32 + lane;
                key[k] = idx[k] = 0;
                if (t >= end) continue;
                // through L2: other SMs wrote the lists
                if (pass) {
                    key[k] = __ldcg(key_in + t);
                    idx[k] = __ldcg(idx_in + t);
                } else {
                    const long long id = index_at(a.ids, a.ids64, t);
                    key[k] = id >= 0 && id < a.V ? static_cast<uint32_t>(id) : static_cast<uint32_t>(a.V);
                    idx[k] = t;
                }
            }
        };
        auto digit = [&](int k) { return (key[k] >> shift) & (nd - 1); };
        // the lanes with a token of the same digit; 0 for a lane without one
        auto match = [&](unsigned t0, int k) {
            const bool on = t0 + k * 32 + lane < end;
            uint32_t same = __ballot_sync(0xffffffffu, on);
            for (int b = 0; b < a.bits; ++b) {
                const bool one = digit(k) >> b & 1;
                const uint32_t ones = __ballot_sync(0xffffffffu, one);
                same &= one ? ones : ~ones;
            }
            return on ? same : 0u;
        };
        load(start);
        for (int i = tid; i < kSortWarps * nd; i += kSortThreads) cnt[i] = 0;
        __syncthreads();
        for (unsigned t0 = start; t0 < end; t0 += 32 * kSortKeep) {
            if (t0 != start) load(t0);
#pragma unroll
            for (int k = 0; k < kSortKeep; ++k) {
                if (t0 + k * 32 >= end) break;  // the whole warp
                peers[k] = match(t0, k);
                if (peers[k] && !(peers[k] & below)) mine[digit(k)] += __popc(peers[k]);
                __syncwarp();
            }
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
        sync_all();
        uint32_t before = 0, sum = 0;
        if (tid < nd) {
#pragma unroll 4
            for (int c = 0; c < nc; ++c) {
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
            uint32_t v = lane < kSortWarps ? wsum[lane] : 0, w = v;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t x = __shfl_up_sync(0xffffffffu, w, o);
                if (lane >= o) w += x;
            }
            if (lane < kSortWarps) wsum[lane] = w - v;
        }
        __syncthreads();
        if (tid < nd) base[tid] = wsum[warp] + inc - sum + before;
        __syncthreads();
        const bool kept = end - start <= 32 * kSortKeep;  // the tokens are still in registers
        for (unsigned t0 = start; t0 < end; t0 += 32 * kSortKeep) {
            if (!kept) load(t0);
#pragma unroll
            for (int k = 0; k < kSortKeep; ++k) {
                if (t0 + k * 32 >= end) break;
                if (!kept) peers[k] = match(t0, k);
                const uint32_t dig = digit(k);
                if (peers[k]) {
                    const uint32_t at = base[dig] + mine[dig] + __popc(peers[k] & below);
                    key_out[at] = key[k];
                    idx_out[at] = idx[k];
                }
                __syncwarp();
                if (peers[k] && !(peers[k] & below)) mine[dig] += __popc(peers[k]);
                __syncwarp();
            }
        }
        // this pass's lists are whole, and nobody reads this CTA's totals any more
        sync_all();
    }
}

// ------------------------------------------------------------------ sums of the sorted rows

constexpr int kGradUnroll = 4;  // rows of a batch; one batch is read ahead

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
__global__ void __launch_bounds__(256, 4) embed_grad_kernel(const EmbedArgs a) {
    using P = Pack<T, N>;
    __shared__ uint32_t skey[256 + 2], sidx[256];
    pdl_wait();
    const unsigned piece0 = blockIdx.x * blockDim.y, S = a.S, n = a.n;
    const uint32_t V = a.V;
    // the block's stretch of the sorted lists, with the ids before and behind it
    const unsigned first = piece0 * S, count = min(n - first, blockDim.y * S);
    for (unsigned i = threadIdx.y * blockDim.x + threadIdx.x; i < count; i += blockDim.x * blockDim.y) {
        skey[i + 1] = a.key[0][first + i];
        sidx[i] = a.idx[0][first + i];
    }
    if (threadIdx.x == 0 && threadIdx.y == 0) {
        skey[0] = first ? a.key[0][first - 1] : ~0u;
        skey[count + 1] = first + count < n ? a.key[0][first + count] : ~0u;
    }
    __syncthreads();
    const unsigned piece = piece0 + threadIdx.y;
    const int unit = blockIdx.y * blockDim.x + threadIdx.x;
    if (piece >= static_cast<unsigned>(a.npieces) || unit * N >= a.D) return;
    const int col = unit * N;
    const unsigned begin = threadIdx.y * S, end = min(begin + S, count);  // of the stretch
    const uint32_t *key = skey + 1;
    const T *dout = static_cast<const T *>(a.dout) + col;
    float *part = a.part + static_cast<size_t>(piece) * 2 * a.Dp + col;

    float s[N];
#pragma unroll
    for (int e = 0; e < N; ++e) s[e] = 0.f;
    uint32_t cur = key[begin];
    bool began = skey[begin] != cur;  // cur's first token lies in this piece
    auto load = [&](P(&v)[kGradUnroll], unsigned i0) {
#pragma unroll
        for (int u = 0; u < kGradUnroll; ++u) {
            const unsigned i = i0 + u;
            v[u] = i < end && key[i] < V ? P::load(dout + sidx[i] * a.ld_dout) : P::zero();
        }
    };
    auto add = [&](const P(&v)[kGradUnroll], unsigned i0) {
#pragma unroll
        for (int u = 0; u < kGradUnroll; ++u) {
            if (i0 + u < end && key[i0 + u] != cur) {
                if (began) {
                    finish<TO, N>(a, cur, col, s);
                } else {
                    store_part<N>(part, s);
                }
                began = true;
                cur = key[i0 + u];
#pragma unroll
                for (int e = 0; e < N; ++e) s[e] = 0.f;
            }
            float f[N];
            v[u].to(f);
#pragma unroll
            for (int e = 0; e < N; ++e) s[e] += f[e];
        }
    };
    P v[kGradUnroll], w[kGradUnroll];
    load(v, begin);
    for (unsigned i0 = begin; i0 < end; i0 += 2 * kGradUnroll) {
        load(w, i0 + kGradUnroll);
        add(v, i0);
        load(v, i0 + 2 * kGradUnroll);
        add(w, i0 + kGradUnroll);
    }
    if (cur >= V) return;  // ids outside the table come last
    const bool more = key[end] == cur;
    if (began && !more) {
        finish<TO, N>(a, cur, col, s);
    } else {
        store_part<N>(part + (began ? a.Dp : 0), s);
        if (began && unit == 0) a.list[atomicAdd(a.count, 1u)] = piece;
    }
}

// The ids that span pieces: for each listed piece p, its partial row 1 plus the rows 0 of the
// pieces that follow while the id goes on, always in the same grouping. A warp takes one of them
// for 32 x 4 columns; those of more than kJoinShort rows are shared by the block's eight warps.
constexpr unsigned kJoinShort = 16;

template <typename TO>
__device__ __forceinline__ void finish_columns(const EmbedArgs &a, uint32_t id, int col, float4 s) {
    const float f[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float one[1] = {f[e]};
        if (col + e < a.D) finish<TO, 1>(a, id, col + e, one);
    }
}

template <typename TO>
__global__ void __launch_bounds__(256) embed_join_kernel(const EmbedArgs a) {
    __shared__ float4 sums[8][32];
    __shared__ unsigned long_piece[8], long_rows[8];
    pdl_wait();
    const int lane = threadIdx.x & 31, y = threadIdx.x >> 5;
    const int col = (blockIdx.y * 32 + lane) * 4;
    const unsigned S = a.S, npieces = a.npieces;
    const uint32_t count = *a.count;
    // rows j0 .. j1 - 1 of piece p's id: row 0 is its partial row 1, row j piece (p + j)'s row 0
    auto rows_sum = [&](unsigned p, unsigned j0, unsigned j1) {
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        if (col < a.Dp) {
#pragma unroll 8
            for (unsigned j = j0; j < j1; ++j) {
                const float4 v = *reinterpret_cast<const float4 *>(
                    a.part + (static_cast<size_t>(p + j) * 2 + (j == 0)) * a.Dp + col);
                s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
            }
        }
        return s;
    };
    for (uint32_t i0 = blockIdx.x * 8; i0 < count; i0 += gridDim.x * 8) {
        unsigned p = 0, rows = 0;
        if (i0 + y < count) {
            p = a.list[i0 + y];
            const uint32_t id = a.key[0][(p + 1) * S - 1];
            for (;;) {  // piece q has some of it when its first token has the id
                const unsigned q = p + 1 + rows + lane;
                const bool has = q < npieces && a.key[0][q * S] == id;
                const uint32_t not_in = ~__ballot_sync(0xffffffffu, has);
                rows += not_in ? __ffs(not_in) - 1 : 32;
                if (not_in) break;
            }
            ++rows;  // and its own
            if (rows <= kJoinShort) finish_columns<TO>(a, id, col, rows_sum(p, 0, rows));
        }
        if (lane == 0) long_piece[y] = p, long_rows[y] = rows > kJoinShort ? rows : 0;
        __syncthreads();
        for (int k = 0; k < 8; ++k) {
            const unsigned m = long_rows[k], q = long_piece[k];
            if (!m) continue;  // the same for the whole block
            const unsigned per = (m + 7) / 8;
            sums[y][lane] = rows_sum(q, min(y * per, m), min((y + 1) * per, m));
            __syncthreads();
            if (y == 0) {
                float4 s = sums[0][lane];
#pragma unroll
                for (int w = 1; w < 8; ++w) {
                    const float4 v = sums[w][lane];
                    s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
                }
                finish_columns<TO>(a, a.key[0][(q + 1) * S - 1], col, s);
            }
            __syncthreads();
        }
        __syncthreads();  // the long ones' lists may be written again
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
    // as many pieces per block as its 256 threads and its stretch of 256 tokens hold
    const int units = a.D / N, tx = units < 256 ? units : 256, fit = 256 / tx, room = 256 / a.S;
    const int ty = fit < room ? fit : room;
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

// CTAs of the sort: a round of 32 tokens costs a warp more than the cluster's barriers do, so one
// round each up to four CTAs, eight for more than 4096 tokens (the whole gradient of 30000 x 768
// bf16 from 8192 tokens: 29.4 us with four, 26.9 with eight; from 16384 tokens 43.8 and 33.9; from
// 4096, 21.0 and 22.8; added to a table, without the zeros' clusters, 26.0 and 22.6, 49.5 and 37.9,
// 19.2 and 17.9). The zeros take the other SMs, or with clusters seven eighths of all (so that every cluster finds its
// place at once: 55 us instead of 62 for a 32768 x 2048 bf16 table).
cudaError_t launch_embed_sort(EmbedArgs a, int bf16_out, int vec, int num_sms, cudaStream_t st) {
    a.sort_ctas = 1;
    while (a.sort_ctas < 4 && a.n > a.sort_ctas * kSortThreads) a.sort_ctas *= 2;
    if (a.n > 4096) a.sort_ctas = 8;
    const int all = a.sort_ctas == 1 ? num_sms : num_sms * 7 / 8 / a.sort_ctas * a.sort_ctas;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.accumulate ? a.sort_ctas : all < 2 * a.sort_ctas ? 2 * a.sort_ctas : all);
    cfg.blockDim = dim3(kSortThreads);
    cfg.dynamicSmemBytes = sort_smem(a.bits);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = a.sort_ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.sort_ctas > 1 ? 2 : 1;
    if (bf16_out)
        return vec ? cudaLaunchKernelEx(&cfg, embed_sort_kernel<__nv_bfloat16, 8>, a)
                   : cudaLaunchKernelEx(&cfg, embed_sort_kernel<__nv_bfloat16, 1>, a);
    return vec ? cudaLaunchKernelEx(&cfg, embed_sort_kernel<float, 4>, a)
               : cudaLaunchKernelEx(&cfg, embed_sort_kernel<float, 1>, a);
}

cudaError_t launch_embed_grad(const EmbedArgs &a, int bf16, int bf16_out, int vec, cudaStream_t st) {
    if (!bf16) return launch_grad_w<float, float>(a, vec, st);
    return bf16_out ? launch_grad_w<__nv_bfloat16, __nv_bfloat16>(a, vec, st)
                    : launch_grad_w<__nv_bfloat16, float>(a, vec, st);
}

cudaError_t launch_embed_join(const EmbedArgs &a, int bf16_out, int num_sms, cudaStream_t st) {
    const int gx = (a.npieces + 7) / 8, most = 2 * num_sms;
    const dim3 grid(gx < most ? gx : most, (a.Dp / 4 + 31) / 32);
    return bf16_out ? launch_pdl(embed_join_kernel<__nv_bfloat16>, grid, dim3(256), 0, st, a)
                    : launch_pdl(embed_join_kernel<float>, grid, dim3(256), 0, st, a);
}

}  // namespace rsa
