// kernels_qknorm.cu -- RMS norm of every head's row of the queries and keys and rotation by its
// position, in one pass, forward and backward (rsa_qk_norm_rope, rsa_rows.h).
//
// Bound by memory: a forward pass reads and writes every element once (2 x 2 bytes in bf16)
// and spends about ten operations on it. A row of d elements lies in the 16-byte vectors of
// d / 8 (bf16) or d / 4 (fp32) neighbouring lanes, so a row's sum is a few shuffles, and the
// other member of a half-split pair is one shuffle of the packed vector away. A tile is P
// consecutive rows of the sequence for all heads of one side (queries or keys): the tile's
// P x rot/2 angles are computed once by the block (fp64 product and reduction, fp32 sine and
// cosine) and every thread keeps the position and columns it serves, so the head loop has the
// cosines, sines and weights in registers and only streams rows.
#include <type_traits>

#include "rows_common.cuh"

namespace rsa {
namespace {

using namespace rows;

constexpr int kThreads = 256;

__device__ __forceinline__ long long position(const QkArgs &a, unsigned b, unsigned l) {
    if (!a.pos) return a.pos0 + l;
    return index_at(a.pos, a.pos64, static_cast<long long>(b) * a.pos_sb + l);
}

// (cos, sin) of position * freq. The angle in turns is formed and reduced in fp64: the product
// of a position below 2^29 with an fp32 frequency is exact, and the reduced turn carries an
// error near 2^-53 of the whole angle.
__device__ __forceinline__ float2 angle(long long pos, float freq) {
    const double turns = static_cast<double>(pos) * static_cast<double>(freq) * 0.15915494309189533577;
    float2 cs;
    sincospif(static_cast<float>(2.0 * (turns - rint(turns))), &cs.y, &cs.x);
    return cs;
}

// A thread's part of the rotation for its VEC columns: y_e = n_e c_e + n_partner(e) s_e, with
// s_e = -sin for the first and +sin for the second member of a pair (columns past rot: 1, 0).
template <int LPR, int VEC, bool INTER>
struct Rotation {
    float c[VEC], s[VEC];

    __device__ __forceinline__ static int partner_lane(int li, int rot) {
        const int nl = rot / 2 / VEC;  // lanes of the half-split pairs' first members
        return INTER || li >= 2 * nl ? li : (li < nl ? li + nl : li - nl);
    }
    __device__ __forceinline__ void load(const float2 *cs, int li, int rot) {
        const int col = li * VEC, half = rot / 2;
        if (INTER) {
#pragma unroll
            for (int e = 0; e < VEC; e += 2) {
                const float2 t = col < rot ? cs[col / 2 + e / 2] : make_float2(1.f, 0.f);
                c[e] = c[e + 1] = t.x;
                s[e] = -t.y, s[e + 1] = t.y;
            }
        } else {
            const bool second = col >= half;
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float2 t =
                    col < rot ? cs[col + e - (second ? half : 0)] : make_float2(1.f, 0.f);
                c[e] = t.x;
                s[e] = second ? t.y : -t.y;
            }
        }
    }
};

// The vector of the pair partners: the neighbouring elements, or the partner lane's vector.
template <int VEC, bool INTER, typename P>
__device__ __forceinline__ void partners(const P &v, const float (&f)[VEC], int lane, float (&g)[VEC]) {
    if constexpr (INTER) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) g[e] = f[e ^ 1];
    } else {
        P w;
        w.raw.x = __shfl_sync(0xffffffffu, v.raw.x, lane);
        w.raw.y = __shfl_sync(0xffffffffu, v.raw.y, lane);
        w.raw.z = __shfl_sync(0xffffffffu, v.raw.z, lane);
        w.raw.w = __shfl_sync(0xffffffffu, v.raw.w, lane);
        w.to(g);
    }
}

template <int LPR>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// The tile's angles: cs[p][i], p < P rows, i < rot / 2.
__device__ __forceinline__ void tile_angles(const QkArgs &a, unsigned m0, unsigned M, float2 *cs) {
    const int half = a.rot / 2, n = half << a.logP;
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const int p = i / half, j = i - p * half;
        const unsigned m = m0 + p;
        if (m < M) {
            const unsigned b = m / a.L;
            cs[i] = angle(position(a, b, m - b * a.L), a.freq[j]);
        }
    }
}

// Forward: grid (tiles of P rows, side). Four rows per thread are in flight.
template <typename T, int LPR, bool INTER>
__global__ void __launch_bounds__(kThreads) qk_norm_kernel(const QkArgs a) {
    constexpr int VEC = 16 / sizeof(T), D = LPR * VEC, R = kThreads / LPR, U = 4;
    using P = Pack<T, VEC>;
    __shared__ float2 cs[R * D / 2];
    pdl_wait();
    const int side = blockIdx.y, H = a.H[side];
    const int li = threadIdx.x % LPR, g = threadIdx.x / LPR;
    const int p = g & ((1 << a.logP) - 1), h0 = g >> a.logP, HG = R >> a.logP;
    const unsigned M = static_cast<unsigned>(a.B) * a.L, m0 = blockIdx.x << a.logP, m = m0 + p;
    const bool live = m < M;
    const unsigned b = live ? m / a.L : 0, l = live ? m - b * a.L : 0;
    const T *x = static_cast<const T *>(a.x[side]) + b * a.sx[side][0] + l * a.sx[side][2] + li * VEC;
    T *y = static_cast<T *>(a.y[side]) + b * a.sy[side][0] + l * a.sy[side][2] + li * VEC;
    const long long hx = a.sx[side][1], hy = a.sy[side][1];

    P v[U];  // the first rows travel while the angles are computed
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int h = h0 + u * HG;
        v[u] = live && h < H ? P::load(x + h * hx) : P::zero();
    }
    tile_angles(a, m0, M, cs);
    __syncthreads();
    // y_e = r (x_e w_e c_e + x_partner w_partner s_e): weights folded into the rotation
    Rotation<LPR, VEC, INTER> rt;
    rt.load(cs + p * (a.rot / 2), li, a.rot);
    const int pl = Rotation<LPR, VEC, INTER>::partner_lane(li, a.rot);
    if (const float *w = a.w[side]) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            rt.c[e] *= w[li * VEC + e];
            rt.s[e] *= w[INTER ? li * VEC + (e ^ 1) : pl * VEC + e];
        }
    }
    const int src = (threadIdx.x & 31 & ~(LPR - 1)) | pl;
    for (int h = h0; h - h0 < H; h += U * HG) {  // the same count for every thread
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float f[VEC], q[VEC], ss = 0.f;
            v[u].to(f);
#pragma unroll
            for (int e = 0; e < VEC; ++e) ss = fmaf(f[e], f[e], ss);
            const float r = rsqrtf(row_sum<LPR>(ss) * (1.f / D) + a.eps);
            partners<VEC, INTER>(v[u], f, src, q);
#pragma unroll
            for (int e = 0; e < VEC; ++e) f[e] = r * fmaf(f[e], rt.c[e], q[e] * rt.s[e]);
            const int hu = h + u * HG, hn = hu + U * HG;
            if (live && hu < H) P::from(f).store(y + hu * hy);
            if (live && hn < H) v[u] = P::load(x + hn * hx);
        }
    }
}

// Backward: persistent blocks, the first nblk[0] on the queries and the rest on the keys, each
// over the tiles of its side; a thread's columns are the same in all of them, so the weights'
// gradient is summed in registers and the block leaves one row of sums in `part`.
template <typename T, int LPR, bool INTER>
__global__ void __launch_bounds__(kThreads) qk_norm_bwd_kernel(const QkArgs a) {
    constexpr int VEC = 16 / sizeof(T), D = LPR * VEC, R = kThreads / LPR, U = 2;
    using P = Pack<T, VEC>;
    __shared__ float2 cs[R * D / 2];  // the sums' exchange at the end: R x D floats
    pdl_wait();
    const int side = blockIdx.x >= a.nblk[0];
    const unsigned blk = blockIdx.x - (side ? a.nblk[0] : 0);
    const int H = a.H[side];
    const int li = threadIdx.x % LPR, g = threadIdx.x / LPR;
    const int p = g & ((1 << a.logP) - 1), h0 = g >> a.logP, HG = R >> a.logP;
    const unsigned M = static_cast<unsigned>(a.B) * a.L, step = 1u << a.logP;
    const long long hx = a.sx[side][1], hy = a.sy[side][1], hd = a.sdy[side][1];
    const int pl = Rotation<LPR, VEC, INTER>::partner_lane(li, a.rot);
    const int src = (threadIdx.x & 31 & ~(LPR - 1)) | pl;
    float w[VEC], dw[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        w[e] = a.w[side] ? a.w[side][li * VEC + e] : 1.f;
        dw[e] = 0.f;
    }
    const unsigned ntiles = (M + step - 1) >> a.logP;
    for (unsigned t = blk; t < ntiles; t += a.nblk[side]) {
        const unsigned m0 = t << a.logP, m = m0 + p;
        const bool live = m < M;
        const unsigned b = live ? m / a.L : 0, l = live ? m - b * a.L : 0;
        const T *x = static_cast<const T *>(a.x[side]) + b * a.sx[side][0] + l * a.sx[side][2] + li * VEC;
        const T *dy = static_cast<const T *>(a.dy[side]) + b * a.sdy[side][0] + l * a.sdy[side][2] + li * VEC;
        T *dx = static_cast<T *>(a.y[side]) + b * a.sy[side][0] + l * a.sy[side][2] + li * VEC;
        P vx[U], vd[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = h0 + u * HG;
            const bool on = live && h < H;
            vx[u] = on ? P::load(x + h * hx) : P::zero();
            vd[u] = on ? P::load(dy + h * hd) : P::zero();
        }
        __syncthreads();  // the previous tile's angles are no longer read
        tile_angles(a, m0, M, cs);
        __syncthreads();
        Rotation<LPR, VEC, INTER> rt;
        if (live) rt.load(cs + p * (a.rot / 2), li, a.rot);
        for (int h = h0; h - h0 < H; h += U * HG) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int hu = h + u * HG, hn = hu + U * HG;
                const bool on = live && hu < H;
                float f[VEC], d[VEC], q[VEC], ss = 0.f, ux = 0.f;
                vx[u].to(f);
                vd[u].to(d);
                partners<VEC, INTER>(vd[u], d, src, q);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    d[e] = fmaf(d[e], rt.c[e], -q[e] * rt.s[e]);  // dn: rotated back
                    ss = fmaf(f[e], f[e], ss);
                    ux = fmaf(d[e] * w[e], f[e], ux);
                }
                ss = row_sum<LPR>(ss);
                ux = row_sum<LPR>(ux);
                const float r = rsqrtf(ss * (1.f / D) + a.eps);
                const float k = r * r * ux * (1.f / D);
                if (on) {
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        dw[e] = fmaf(d[e], f[e] * r, dw[e]);
                        d[e] = r * fmaf(d[e], w[e], -f[e] * k);
                    }
                    P::from(d).store(dx + hu * hy);
                }
                if (live && hn < H) {
                    vx[u] = P::load(x + hn * hx);
                    vd[u] = P::load(dy + hn * hd);
                }
            }
        }
    }
    if (!a.part) return;
    // the block's sums: R row groups over D columns, added in a fixed order
    float *sum = reinterpret_cast<float *>(cs);
    __syncthreads();
#pragma unroll
    for (int e = 0; e < VEC; ++e) sum[g * D + li * VEC + e] = dw[e];
    __syncthreads();
    if (threadIdx.x < D) {
        float s = 0.f;
        for (int i = 0; i < R; ++i) s += sum[i * D + threadIdx.x];
        a.part[static_cast<size_t>(blockIdx.x) * D + threadIdx.x] = s;
    }
}

// dw[side][col] = sum over the side's blocks of their sums: grid (d / 32, side), 32 columns x
// 8 slices of the blocks.
__global__ void __launch_bounds__(256) qk_dw_kernel(const QkArgs a) {
    __shared__ float sum[8][32];
    pdl_wait();
    const int side = blockIdx.y, col = blockIdx.x * 32 + (threadIdx.x & 31), y = threadIdx.x >> 5;
    const int first = side ? a.nblk[0] : 0, n = a.nblk[side];
    float s = 0.f;
    for (int i = y; i < n; i += 8) s += a.part[static_cast<size_t>(first + i) * a.d + col];
    sum[y][threadIdx.x & 31] = s;
    __syncthreads();
    if (y == 0 && a.dw[side]) {
        s = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) s += sum[i][threadIdx.x];
        a.dw[side][col] = s;
    }
}

template <typename T, int LPR, bool INTER>
cudaError_t launch(const QkArgs &a, int backward, cudaStream_t st) {
    const unsigned M = static_cast<unsigned>(a.B) * a.L;
    const unsigned tiles = (M + (1u << a.logP) - 1) >> a.logP;
    if (backward)
        return launch_pdl(qk_norm_bwd_kernel<T, LPR, INTER>, dim3(a.nblk[0] + a.nblk[1]),
                          dim3(kThreads), 0, st, a);
    return launch_pdl(qk_norm_kernel<T, LPR, INTER>, dim3(tiles, 2), dim3(kThreads), 0, st, a);
}

template <typename T, int LPR>
cudaError_t launch_i(const QkArgs &a, int backward, cudaStream_t st) {
    return a.inter ? launch<T, LPR, true>(a, backward, st) : launch<T, LPR, false>(a, backward, st);
}

// Rows per tile: the most, up to the row groups of a block, that still leave `want` tiles.
int tile_log(unsigned M, int groups, unsigned want) {
    int k = 0;
    while ((2 << k) <= groups && ((M >> (k + 1)) >= want)) ++k;
    return k;
}

}  // namespace

// Blocks of the backward kernel: four per SM, shared between the sides in the proportion of
// their heads, at least one each.
cudaError_t launch_qk_norm(QkArgs &a, int backward, int bf16, int num_sms, cudaStream_t st) {
    const int vec = bf16 ? 8 : 4, lpr = a.d / vec, groups = kThreads / lpr;
    const unsigned M = static_cast<unsigned>(a.B) * a.L;
    a.logP = tile_log(M, groups, 4u * num_sms);
    if (backward) {
        const int total = kQkBlocksPerSm * (num_sms < kQkMaxSms ? num_sms : kQkMaxSms);
        int nq = static_cast<int>(static_cast<long long>(total) * a.H[0] / (a.H[0] + a.H[1]));
        nq = nq < 1 ? 1 : nq > total - 1 ? total - 1 : nq;
        const unsigned tiles = (M + (1u << a.logP) - 1) >> a.logP;
        a.nblk[0] = static_cast<unsigned>(nq) < tiles ? nq : static_cast<int>(tiles);
        a.nblk[1] = static_cast<unsigned>(total - nq) < tiles ? total - nq : static_cast<int>(tiles);
    }
    if (bf16) {
        switch (a.d) {
            case 32: return launch_i<__nv_bfloat16, 4>(a, backward, st);
            case 64: return launch_i<__nv_bfloat16, 8>(a, backward, st);
            default: return launch_i<__nv_bfloat16, 16>(a, backward, st);
        }
    }
    switch (a.d) {
        case 32: return launch_i<float, 8>(a, backward, st);
        case 64: return launch_i<float, 16>(a, backward, st);
        default: return launch_i<float, 32>(a, backward, st);
    }
}

cudaError_t launch_qk_dw(const QkArgs &a, cudaStream_t st) {
    return launch_pdl(qk_dw_kernel, dim3(a.d / 32, 2), dim3(256), 0, st, a);
}

}  // namespace rsa
