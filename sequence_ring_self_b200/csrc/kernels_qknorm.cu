// kernels_qknorm.cu -- RMS norm of every head's row of the queries and keys and rotation by its
// position, in one pass, forward and backward (rsa_qk_norm_rope, rsa_rows.h).
//
// Bound by memory: a forward pass reads and writes every element once (2 x 2 bytes in bf16)
// and spends about ten operations on it, a backward pass three times and twenty. Rows are held
// in 16-byte vectors by neighbouring lanes, so that a row's sums are a few shuffles. A tile is P
// consecutive rows of the sequence for all heads of one side (queries or keys): the tile's angles
// are computed once by the block (fp64 product and reduction, fp32 sine and cosine) and a thread
// keeps the row and columns it serves, so the head loop only streams rows.
#include <type_traits>

#include "rows_common.cuh"

namespace rsa {
namespace {

using namespace rows;

constexpr int kThreads = 256;
// 1 / root mean square of a row of large numbers; others' products overflow with weights past 2^100
constexpr float kLargeRow = 0x1p-20f;

__device__ __forceinline__ long long position(const QkArgs &a, unsigned b, unsigned l) {
    if (!a.pos) return a.pos0 + l;
    return index_at(a.pos, a.pos64, static_cast<long long>(b) * a.pos_sb + l);
}

__device__ __forceinline__ double turns_per_unit(long long pos) {
    return static_cast<double>(pos) * 0.15915494309189533577;  // 1 / 2 pi
}

// (cos, sin) of position * freq, pos = position / 2 pi. The angle in turns is formed and reduced
// in fp64: three roundings of 2^-53 of the whole angle (1 / 2 pi and two products), and one of the
// reduced angle to fp32.
__device__ __forceinline__ float2 angle(double pos, float freq) {
    const double turns = pos * static_cast<double>(freq);
    float2 cs;
    sincospif(static_cast<float>(2.0 * (turns - rint(turns))), &cs.y, &cs.x);
    return cs;
}

// Backward: a row of D = 2 LPR VEC elements is held by LPR lanes, two vectors each: the pairs' first and
// second members where half-split pairs are rotated (the first rot / 2 / VEC lanes; the others
// share the vectors behind rot), halves of the row with neighbouring pairs.
template <int LPR, int VEC, bool INTER>
__device__ __forceinline__ void lane_columns(int t, int rot, int (&col)[2]) {
    const int nl = INTER ? 0 : rot / 2 / VEC;
    if (t < nl)
        col[0] = t, col[1] = t + nl;
    else
        col[0] = t + nl, col[1] = t + LPR;
    col[0] *= VEC, col[1] *= VEC;
}

// Rotation factors, VEC pairs per lane: pair j of the row lies at factor_at(j) of each of the
// tile row's three lists of D / 2 numbers: cos, sin, -sin. Pairs behind rot / 2 have (1, 0, 0).
// Neighbouring lanes' four-number accesses are neighbours: a warp's read has no bank conflict.
template <int LPR, int VEC, bool INTER>
__device__ __forceinline__ int factor_at(int j) {
    int t = j / VEC, e = j % VEC;
    if (INTER) {  // VEC / 2 pairs of each of the lane's vectors
        const int v = j / (VEC / 2);
        t = v % LPR, e = j % (VEC / 2) + v / LPR * (VEC / 2);
    }
    return e / 4 * (LPR * 4) + t * 4 + e % 4;
}

// The block fills cs[p][3][D / 2] for the tile's rows p < P, each row by 256 / P threads.
template <int LPR, int VEC, bool INTER>
__device__ __forceinline__ void tile_factors(const QkArgs &a, unsigned m0, unsigned M, float *cs) {
    constexpr int N = LPR * VEC;  // pairs of a row
    const int per = kThreads >> a.logP, p = threadIdx.x / per, half = a.rot / 2;
    const unsigned m = m0 + p;
    if (m >= M) return;
    const unsigned b = m / a.L;
    const double pos = turns_per_unit(position(a, b, m - b * a.L));
    float *row = cs + p * 3 * N;
    for (int j = threadIdx.x & (per - 1); j < N; j += per) {
        const float2 t = j < half ? angle(pos, a.freq[j]) : make_float2(1.f, 0.f);
        const int at = factor_at<LPR, VEC, INTER>(j);
        row[at] = t.x;
        row[N + at] = t.y;
        row[2 * N + at] = -t.y;
    }
}

// The same for one number per column, VEC columns per lane.
template <int LPR, int VEC>
__device__ __forceinline__ int column_at(int col) {
    return col % VEC / 4 * (LPR * 4) + col / VEC * 4 + col % 4;
}

// A lane's VEC numbers of one list.
template <int LPR, int VEC>
__device__ __forceinline__ void load_factors(const float *list, int t, float2 (&f)[VEC / 2]) {
#pragma unroll
    for (int e = 0; e < VEC; e += 4) {
        const float4 v = *reinterpret_cast<const float4 *>(list + e * LPR + t * 4);
        f[e / 2] = make_float2(v.x, v.y);
        f[e / 2 + 1] = make_float2(v.z, v.w);
    }
}

// With neighbouring pairs, pair i of vector k of the lane: its number of a list of VEC.
template <int VEC>
__device__ __forceinline__ float of_pair(const float2 (&f)[VEC / 2], int k, int i) {
    const int n = k * (VEC / 2) + i;
    return n & 1 ? f[n / 2].y : f[n / 2].x;
}

__device__ __forceinline__ float2 swapped(float2 v) { return make_float2(v.y, v.x); }

template <int LPR>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// VEC weights from a column on, in pairs, by way of shared memory (the caller's array need not
// be aligned for vector loads).
template <int VEC>
__device__ __forceinline__ void load_weights(const float *sw, int col, float2 (&w)[VEC / 2]) {
#pragma unroll
    for (int e = 0; e < VEC / 2; ++e) w[e] = reinterpret_cast<const float2 *>(sw + col)[e];
}

// Forward: grid (tiles of P rows, side); one vector of a row per lane, LPR lanes per row, four rows
// per thread in flight. With the weights folded in, a column has two factors,
//   y_e = r (x_e f_e + x_partner(e) g_e),
// which the block leaves in shared memory for the tile's rows and a thread keeps for its own.
// The partner's vector comes by shuffles of the packed one: against two vectors per thread
// (as in the backward pass) this has more instructions, but whole 128-byte rows per access at
// d = 64 and more blocks per SM: 28.1 us against 37.2 for 4 x 4096 rows of 16 + 16 heads of 64.
template <typename T, int LPR, bool INTER>
__global__ void __launch_bounds__(kThreads) qk_norm_kernel(const QkArgs a) {
    constexpr int VEC = 16 / sizeof(T), D = LPR * VEC, R = kThreads / LPR, U = 4, E = VEC / 2;
    using P = Pack<T, VEC>;
    __shared__ __align__(16) float cs[R * 2 * D];  // [p][f, g][D]
    pdl_wait();
    const int side = blockIdx.y, H = a.H[side];
    const int t = threadIdx.x % LPR, g = threadIdx.x / LPR;
    const int p = g & ((1 << a.logP) - 1), h0 = g >> a.logP, HG = R >> a.logP;
    const unsigned M = static_cast<unsigned>(a.B) * a.L, m0 = blockIdx.x << a.logP, m = m0 + p;
    const bool live = m < M;
    const unsigned b = live ? m / a.L : 0, l = live ? m - b * a.L : 0;
    const long long hx = a.sx[side][1] * HG, hy = a.sy[side][1] * HG;  // to the next round's head
    const T *x = static_cast<const T *>(a.x[side]) + b * a.sx[side][0] + l * a.sx[side][2] +
                 a.sx[side][1] * h0 + t * VEC;
    T *y = static_cast<T *>(a.y[side]) + b * a.sy[side][0] + l * a.sy[side][2] +
           a.sy[side][1] * h0 + t * VEC;
    const int left = live && h0 < H ? (H - h0 + HG - 1) / HG : 0;  // this thread's rows

    P v[U];  // the first rows travel while the angles are computed
#pragma unroll
    for (int u = 0; u < U; ++u, x += hx) v[u] = u < left ? P::load(x) : P::zero();
    {
        const int per = kThreads >> a.logP, q = threadIdx.x / per, half = a.rot / 2;
        const unsigned mq = m0 + q;
        if (mq < M) {
            const unsigned bq = mq / a.L;
            const double pos = turns_per_unit(position(a, bq, mq - bq * a.L));
            const float *w = a.w[side];
            float *row = cs + q * 2 * D;
            for (int j = threadIdx.x & (per - 1); j < D / 2; j += per) {
                const float2 cj = j < half ? angle(pos, a.freq[j]) : make_float2(1.f, 0.f);
                // the pair's columns; behind rot two that are left as they are
                const int c0 = INTER || j >= half ? 2 * j : j, c1 = INTER || j >= half ? c0 + 1 : j + half;
                const float w0 = w ? w[c0] : 1.f, w1 = w ? w[c1] : 1.f;
                const int u = column_at<LPR, VEC>(c0), z = column_at<LPR, VEC>(c1);
                row[u] = cj.x * w0, row[z] = cj.x * w1;
                row[D + u] = -cj.y * w1, row[D + z] = cj.y * w0;
            }
        }
    }
    __syncthreads();
    float2 f0[E], f1[E];
    load_factors<LPR, VEC>(cs + p * 2 * D, t, f0);
    load_factors<LPR, VEC>(cs + p * 2 * D + D, t, f1);
    const int nl = a.rot / 2 / VEC;  // lanes of the half-split pairs' first members
    const int partner = t < nl ? t + nl : t < 2 * nl ? t - nl : t;
    const int src = (threadIdx.x & 31 & ~(LPR - 1)) | partner;
    for (int i = 0; i * HG < H; i += U) {  // the same count for every thread
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float2 f[E], q[E], ss = make_float2(0.f, 0.f);
            v[u].to(f);
#pragma unroll
            for (int e = 0; e < E; ++e) ss = fma2(f[e], f[e], ss);
            float2 r = both(rsqrtf(row_sum<LPR>(ss.x + ss.y) * (1.f / D) + a.eps));
            // Large numbers take r first, since their products with the factors might overflow (all
            // the more where their squares did, and r = 0). Neighbouring pairs always do; where the
            // partner's vector would have to be scaled too, only a row of large numbers does (for every
            // row: 8.4 us instead of 7.7 for 2048 rows of 16 + 16 heads of 128).
            if (INTER) {
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const float2 n = mul2(f[e], r);
                    f[e] = fma2(n, f0[e], mul2(swapped(n), f1[e]));
                }
            } else {
                P w;
                w.raw.x = __shfl_sync(0xffffffffu, v[u].raw.x, src);
                w.raw.y = __shfl_sync(0xffffffffu, v[u].raw.y, src);
                w.raw.z = __shfl_sync(0xffffffffu, v[u].raw.z, src);
                w.raw.w = __shfl_sync(0xffffffffu, v[u].raw.w, src);
                w.to(q);
                if (r.x < kLargeRow) {
#pragma unroll
                    for (int e = 0; e < E; ++e) f[e] = mul2(f[e], r), q[e] = mul2(q[e], r);
                    r = both(1.f);
                }
#pragma unroll
                for (int e = 0; e < E; ++e) f[e] = mul2(r, fma2(f[e], f0[e], mul2(q[e], f1[e])));
            }
            if (i + u < left) P::from(f).store(y);
            if (i + u + U < left) v[u] = P::load(x);
            x += hx;
            y += hy;
        }
    }
}

// Backward: persistent blocks, the first nblk[0] on the queries and the rest on the keys, each
// over the tiles of its side; a thread's columns are the same in all of them, so the weights'
// gradient is summed in registers and the block leaves one row of sums in `part`. Rows travel
// through kStages slots of each thread by asynchronous copies, two rows ahead and across
// tiles; the factors of the next tile are computed while this one's rows arrive. Both members of
// a pair are the thread's own: with one vector per thread and the partner's fetched by shuffles
// the kernel was bound by its instructions (86 us instead of 70 for 16384 rows of 16 + 16 heads of
// 128, bf16: 402 MB, 88% of a copy's rate).
constexpr int kStages = 3;

template <typename T, int LPR, bool INTER>
__global__ void __launch_bounds__(kThreads, kQkBlocksPerSm) qk_norm_bwd_kernel(const QkArgs a) {
    constexpr int VEC = 16 / sizeof(T), N = LPR * VEC, D = 2 * N, R = kThreads / LPR, E = VEC / 2;
    using P = Pack<T, VEC>;
    extern __shared__ __align__(16) uint8_t dyn[];
    uint4(*slots)[4][kThreads] = reinterpret_cast<uint4(*)[4][kThreads]>(dyn);  // [stage][x0 x1 dy0 dy1]
    float *factors = reinterpret_cast<float *>(dyn + sizeof(uint4) * kStages * 4 * kThreads);
    __shared__ __align__(16) float sw[D];
    pdl_trigger();  // the kernel that adds the weights' gradients up may take its place
    pdl_wait();
    const int side = blockIdx.x >= a.nblk[0], tid = threadIdx.x;
    const unsigned blk = blockIdx.x - (side ? a.nblk[0] : 0);
    const int H = a.H[side];
    const int tl = tid % LPR, g = tid / LPR;
    const int p = g & ((1 << a.logP) - 1), h0 = g >> a.logP, HG = R >> a.logP;
    const int rounds = (H + HG - 1) / HG, size = 3 * N << a.logP;
    const unsigned M = static_cast<unsigned>(a.B) * a.L;
    const unsigned ntiles = (M + (1u << a.logP) - 1) >> a.logP, nblk = a.nblk[side];
    const int mine = h0 < H ? (H - h0 + HG - 1) / HG : 0;  // this thread's rounds
    int col[2];
    lane_columns<LPR, VEC, INTER>(tl, a.rot, col);
    // to the next round's head, and from a tile row to the thread's first one
    const long long hx = a.sx[side][1] * HG, hy = a.sy[side][1] * HG, hd = a.sdy[side][1] * HG;
    const long long first_x = a.sx[side][1] * h0, first_y = a.sy[side][1] * h0,
                    first_d = a.sdy[side][1] * h0;

    // the row to be fetched next: tile, round, and its address
    unsigned ft = blk;
    int fr = 0;
    const T *fx = nullptr, *fd = nullptr;
    auto fetch = [&](int stage) {
        if (ft < ntiles) {
            const unsigned m = (ft << a.logP) + p;
            if (m < M) {
                if (fr == 0) {
                    const unsigned b = m / a.L, l = m - b * a.L;
                    fx = static_cast<const T *>(a.x[side]) + b * a.sx[side][0] + l * a.sx[side][2] + first_x;
                    fd = static_cast<const T *>(a.dy[side]) + b * a.sdy[side][0] + l * a.sdy[side][2] + first_d;
                }
                if (fr < mine) {
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        cp_async16(&slots[stage][k][tid], fx + col[k]);
                        cp_async16(&slots[stage][2 + k][tid], fd + col[k]);
                    }
                }
                fx += hx;
                fd += hd;
            }
            if (++fr == rounds) fr = 0, ft += nblk;
        }
        cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) fetch(i);
    if (tid < D) sw[tid] = a.w[side] ? a.w[side][tid] : 1.f;
    tile_factors<LPR, VEC, INTER>(a, blk << a.logP, M, factors);
    __syncthreads();
    float2 w[2][E], dw[2][E];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        load_weights<VEC>(sw, col[k], w[k]);
#pragma unroll
        for (int e = 0; e < E; ++e) dw[k][e] = make_float2(0.f, 0.f);
    }
    int stage = 0, buf = 0;
    for (unsigned t = blk; t < ntiles; t += nblk) {
        if (t + nblk < ntiles)
            tile_factors<LPR, VEC, INTER>(a, (t + nblk) << a.logP, M, factors + (buf ^ 1) * size);
        const float *row = factors + buf * size + p * 3 * N;
        const unsigned m = (t << a.logP) + p;
        const bool live = m < M;
        const unsigned b = live ? m / a.L : 0, l = live ? m - b * a.L : 0;
        T *dx = static_cast<T *>(a.y[side]) + b * a.sy[side][0] + l * a.sy[side][2] + first_y;
        for (int i = 0; i < rounds; ++i, dx += hy) {
            fetch((stage + kStages - 1) % kStages);
            cp_async_wait<kStages - 1>();
            // rows past the end read a slot's old contents: they stay among their own lanes and
            // nothing of them is kept
            P v[2];
            float2 d[2][E], f[2][E], c[E], s[E];
            v[0].raw = slots[stage][2][tid];
            v[1].raw = slots[stage][3][tid];
            v[0].to(f[0]);
            v[1].to(f[1]);
            load_factors<LPR, VEC>(row, tl, c);
            load_factors<LPR, VEC>(row + N, tl, s);
            // dn, rotated back
            if (INTER) {
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        const float se = of_pair<VEC>(s, k, e);
                        d[k][e] = fma2(swapped(f[k][e]), make_float2(se, -se),
                                       mul2(f[k][e], both(of_pair<VEC>(c, k, e))));
                    }
            } else {
#pragma unroll
                for (int e = 0; e < E; ++e) d[0][e] = fma2(f[1][e], s[e], mul2(f[0][e], c[e]));
                load_factors<LPR, VEC>(row + 2 * N, tl, s);
#pragma unroll
                for (int e = 0; e < E; ++e) d[1][e] = fma2(f[0][e], s[e], mul2(f[1][e], c[e]));
            }
            v[0].raw = slots[stage][0][tid];
            v[1].raw = slots[stage][1][tid];
            v[0].to(f[0]);
            v[1].to(f[1]);
            stage = (stage + 1) % kStages;
            float2 ss[2], ux[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                ss[k] = ux[k] = make_float2(0.f, 0.f);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    ss[k] = fma2(f[k][e], f[k][e], ss[k]);
                    ux[k] = fma2(mul2(d[k][e], w[k][e]), f[k][e], ux[k]);
                }
            }
            ss[0] = add2(ss[0], ss[1]);
            ux[0] = add2(ux[0], ux[1]);
            const float s1 = row_sum<LPR>(ss[0].x + ss[0].y), s2 = row_sum<LPR>(ux[0].x + ux[0].y);
            const float r = rsqrtf(s1 * (1.f / D) + a.eps);
            float q = -r * (r * s2) * (1.f / D);  // (r s2 is of the size of u, r r need not be finite)
            // Numbers so large that s2 overflowed (and r may be 0): the sum once more, of r x. The
            // shuffles are the whole warp's (by the row's lanes alone, in a branch of their own: 75 us
            // instead of 70), the result is taken by the rows concerned.
            const bool over = !(fabsf(s2) < INFINITY);
            if (__builtin_expect(__any_sync(0xffffffffu, over), 0)) {
                float2 v2 = make_float2(0.f, 0.f);
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int e = 0; e < E; ++e)
                        v2 = fma2(mul2(d[k][e], w[k][e]), mul2(f[k][e], both(r)), v2);
                const float s3 = row_sum<LPR>(v2.x + v2.y);
                if (over) q = -r * s3 * (1.f / D);
            }
            if (live && i < mine) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        f[k][e] = mul2(f[k][e], both(r));
                        dw[k][e] = fma2(d[k][e], f[k][e], dw[k][e]);
                        // r (u - x r^2 mean(u x)), u = dn w
                        d[k][e] = fma2(f[k][e], both(q), mul2(mul2(d[k][e], w[k][e]), both(r)));
                    }
                    P::from(d[k]).store(dx + col[k]);
                }
            }
        }
        __syncthreads();  // the factors: this tile's are done with, the next one's are there
        buf ^= 1;
    }
    if (!a.part) return;
    // the block's sums: R row groups over D columns, added in a fixed order
    float *sum = reinterpret_cast<float *>(dyn);
    cp_async_wait<0>();
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int e = 0; e < E; ++e)
            reinterpret_cast<float2 *>(sum + g * D + col[k])[e] = dw[k][e];
    __syncthreads();
    if (tid < D) {
        float s = 0.f;
        for (int i = 0; i < R; ++i) s += sum[i * D + tid];
        a.part[static_cast<size_t>(blockIdx.x) * D + tid] = s;
    }
}

// dw[side][col] = sum over the side's blocks of their sums: grid (d / 32, side), 32 columns x
// 32 slices of the blocks.
__global__ void __launch_bounds__(1024) qk_dw_kernel(const QkArgs a) {
    __shared__ float sum[32][33];
    pdl_wait();
    const int side = blockIdx.y, lane = threadIdx.x & 31, y = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + lane;
    const int first = side ? a.nblk[0] : 0, n = a.nblk[side];
    float s = 0.f;
#pragma unroll 8
    for (int i = y; i < n; i += 32) s += a.part[static_cast<size_t>(first + i) * a.d + col];
    sum[y][lane] = s;
    __syncthreads();
    if (!a.dw[side]) return;
    s = sum[lane][y];  // slice `lane` of column y
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) a.dw[side][blockIdx.x * 32 + y] = s;
}

size_t bwd_smem(int d, int logP) {
    return sizeof(uint4) * kStages * 4 * kThreads + size_t(4) * 2 * (3 * d / 2 << logP);
}

template <typename T, int LPR, bool INTER>
cudaError_t launch(const QkArgs &a, int backward, cudaStream_t st) {
    const unsigned M = static_cast<unsigned>(a.B) * a.L;
    const unsigned tiles = (M + (1u << a.logP) - 1) >> a.logP;
    if (backward)
        return launch_pdl(qk_norm_bwd_kernel<T, LPR, INTER>, dim3(a.nblk[0] + a.nblk[1]),
                          dim3(kThreads), bwd_smem(a.d, a.logP), st, a);
    return launch_pdl(qk_norm_kernel<T, 2 * LPR, INTER>, dim3(tiles, 2), dim3(kThreads), 0, st, a);
}

template <typename T, int LPR>
cudaError_t launch_i(const QkArgs &a, int backward, cudaStream_t st) {
    return a.inter ? launch<T, LPR, true>(a, backward, st) : launch<T, LPR, false>(a, backward, st);
}

// Rows per tile (as a power of two): the most, up to `most`, that still leave `want` tiles.
int tile_log(unsigned M, int most, unsigned want) {
    int k = 0;
    while ((2 << k) <= most && ((M >> (k + 1)) >= want)) ++k;
    return k;
}

template <typename T, int LPR>
cudaError_t configure() {
    const int smem = static_cast<int>(bwd_smem(LPR * 32 / sizeof(T), kQkMaxLogP));
    const cudaError_t e = cudaFuncSetAttribute(qk_norm_bwd_kernel<T, LPR, false>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    return e != cudaSuccess ? e
                            : cudaFuncSetAttribute(qk_norm_bwd_kernel<T, LPR, true>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
}

}  // namespace

// Tiles of as many rows as leave every SM one: a tile's angles cost more than uneven ends do
// (four tiles per SM: 13.8 us instead of 8.2 for 2048 rows of 16 + 16 heads of 128, forward; two
// per SM: 15.2 instead of 10.4 for 2331 rows of 6 + 2 heads of 64, fp32, backward). The backward
// pass takes at most 2^kQkMaxLogP rows, so that its blocks end together (32 rows: 77 us instead
// of 70 for 16384 rows of 16 + 16 heads of 128), in kQkBlocksPerSm blocks per SM shared between
// the sides in the proportion of their heads, at least one each.
cudaError_t launch_qk_norm(QkArgs &a, int backward, int bf16, int num_sms, cudaStream_t st) {
    const int vec = bf16 ? 8 : 4, lpr = a.d / (2 * vec), groups = kThreads / lpr;
    const unsigned M = static_cast<unsigned>(a.B) * a.L;
    if (backward) {
        const int most = groups < (1 << kQkMaxLogP) ? groups : 1 << kQkMaxLogP;
        a.logP = tile_log(M, most, num_sms);
        const int total = kQkBlocksPerSm * (num_sms < kQkMaxSms ? num_sms : kQkMaxSms);
        int nq = static_cast<int>(static_cast<long long>(total) * a.H[0] / (a.H[0] + a.H[1]));
        nq = nq < 1 ? 1 : nq > total - 1 ? total - 1 : nq;
        const unsigned tiles = (M + (1u << a.logP) - 1) >> a.logP;
        a.nblk[0] = static_cast<unsigned>(nq) < tiles ? nq : static_cast<int>(tiles);
        a.nblk[1] = static_cast<unsigned>(total - nq) < tiles ? total - nq : static_cast<int>(tiles);
    } else {
        a.logP = tile_log(M, groups / 2, num_sms);
    }
    if (bf16) {
        switch (a.d) {
            case 32: return launch_i<__nv_bfloat16, 2>(a, backward, st);
            case 64: return launch_i<__nv_bfloat16, 4>(a, backward, st);
            default: return launch_i<__nv_bfloat16, 8>(a, backward, st);
        }
    }
    switch (a.d) {
        case 32: return launch_i<float, 4>(a, backward, st);
        case 64: return launch_i<float, 8>(a, backward, st);
        default: return launch_i<float, 16>(a, backward, st);
    }
}

cudaError_t launch_qk_dw(const QkArgs &a, cudaStream_t st) {
    return launch_pdl(qk_dw_kernel, dim3(a.d / 32, 2), dim3(1024), 0, st, a);
}

cudaError_t qk_kernels_configure() {
    cudaError_t e;
    if ((e = configure<__nv_bfloat16, 2>()) != cudaSuccess ||
        (e = configure<__nv_bfloat16, 4>()) != cudaSuccess ||
        (e = configure<__nv_bfloat16, 8>()) != cudaSuccess ||
        (e = configure<float, 4>()) != cudaSuccess || (e = configure<float, 8>()) != cudaSuccess)
        return e;
    return configure<float, 16>();
}

}  // namespace rsa
