// Irreps norm: lane k of L holds the channel vectors k, k + L, ... (CG of them) of each of a block's
// M = 2l + 1 rows, all loads of a segment in flight together. Where a row of channels is MV < L vectors
// (8 channels), the L lanes lie along the block's rows one after another instead, so that they read
// 128 bytes in one piece (100,000 x 16 rows: forward 17 us against 20 with two lanes a row, backward
// without the parameters 26 against 31); a lane's channels are the vector k modulo MV.
//
// Memory is read 128 bytes at a time, so that the end of a block's rows brings some of the next
// block's: loads that let the caches keep those (forward, 500,000 x 9 x 16: 110, 99 us; 1,000,000 x 9
// x 7: 165, 123 us; wide rows the same either way).
//
// Bound by memory from 16 channels on. Forward, a node's blocks one after another: its rows are read
// and written as one stretch (64,000 x 31 x 128 fp32: 325 us, 93% of the copy rate; blocks taken
// apart by thread blocks of their own reached 66%). Backward, one block of a tile of nodes at a time,
// so that a lane's sums of dw and db stay in registers meanwhile; behind the tile they are added to
// the thread's own sums in shared memory. Few nodes a tile, so that the next block's entries are still
// in the caches (500,000 x 9 x 16: 187 us with all nodes as one tile, 803 MB read where x and dy hold 576;
// 150 us in tiles; 1,000,000 x 9 x 7: 400 and 185 us; 64,000 x 31 x 128 bf16 252 and 243). With rows
// of whole 128 bytes one tile is as good or better (64,000 x 31 x 128 fp32: 478 us, 94%, in tiles 504).
#pragma once
#include "norm.cuh"
#include "norm_segments.cuh"

namespace e3gb {
namespace blocks {

using segments::group_sum;
using segments::RawT;
using segments::store;
using segments::unpack;

template <class T, int VEC, bool KEEP>
__device__ __forceinline__ RawT<T, VEC> load_raw(const T* p, bool ok) {   // KEEP: its neighbours are read next
    RawT<T, VEC> r{};
    const auto* q = reinterpret_cast<const RawT<T, VEC>*>(p);
    if (ok) r = KEEP ? *q : __ldcs(q);
    return r;
}

// where a lane's kRows x CG vectors of a block of M rows lie
template <int VEC, int L, int MV, int CG, int M>
struct Place {
    static constexpr bool kAlong = MV < L;
    static constexpr int kRows = kAlong ? (M * MV + L - 1) / L : M;
    int lane, mul, vecs;
    __device__ __forceinline__ Place(int lane_, int mul_) : lane(lane_), mul(mul_), vecs(mul_ / VEC) {}
    __device__ __forceinline__ int first() const { return lane * VEC; }
    __device__ __forceinline__ int entry(int m, int c) const {   // behind the first
        return kAlong ? m * L * VEC : m * mul + c * L * VEC;
    }
    __device__ __forceinline__ bool in(int m, int c) const {
        return kAlong ? lane + m * L < M * vecs : lane + c * L < vecs;
    }
    __device__ __forceinline__ bool has_channel(int c) const { return kAlong || lane + c * L < vecs; }
    __device__ __forceinline__ int channel(int c) const {   // of the first of vector c's
        return kAlong ? (lane & (vecs - 1)) * VEC : (lane + c * L) * VEC;
    }
};

template <int L>
struct BlockLanes {
    static constexpr int kPerBlock = 256 / L;   // nodes that a thread block takes at a time
    int lane = threadIdx.x % L;
    int64_t step = int64_t(gridDim.x) * kPerBlock;
};

// block b of U nodes, the first of them n0 and kPerBlock apart
template <class TX, class TY, int VEC, int L, int MV, int CG, int M, int U, bool KEEP>
__device__ __forceinline__ void block_forward(const NormShape& sh, int b, int64_t n0, int lane, const TX* x,
                                              const float* w, const float* bias, float eps, TY* y, float2* stats) {
    using P = Place<VEC, L, MV, CG, M>;
    const int mul = int(sh.mul);
    const P at(lane, mul);
    const bool centred = sh.scalar[b] >= 0;
    const int row0 = sh.first_row[b] * mul + at.first();
    RawT<TX, VEC> raw[U][P::kRows][CG];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t n = n0 + u * BlockLanes<L>::kPerBlock;
        const TX* xs = x + (n * sh.x_stride + row0);
#pragma unroll
        for (int m = 0; m < P::kRows; ++m)
#pragma unroll
            for (int c = 0; c < CG; ++c) raw[u][m][c] = load_raw<TX, VEC, KEEP>(xs + at.entry(m, c), n < sh.rows && at.in(m, c));
    }
    const float inv = 1.f / float(M * mul);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t n = n0 + u * BlockLanes<L>::kPerBlock;
        TY* ys = y + (n * sh.x_stride + row0);
        float f[P::kRows][CG][VEC], mu = 0.f, sq = 0.f;
#pragma unroll
        for (int m = 0; m < P::kRows; ++m)
#pragma unroll
            for (int c = 0; c < CG; ++c) unpack(raw[u][m][c], f[m][c]);
        if (M == 1 && centred) {
#pragma unroll
            for (int c = 0; c < CG; ++c)
#pragma unroll
                for (int k = 0; k < VEC; ++k) mu += f[0][c][k];
            mu = group_sum<L>(mu, nullptr) * inv;
        }
#pragma unroll
        for (int m = 0; m < P::kRows; ++m)
#pragma unroll
            for (int c = 0; c < CG; ++c)
#pragma unroll
                for (int k = 0; k < VEC; ++k) {
                    if (M == 1) f[m][c][k] = at.in(m, c) ? f[m][c][k] - mu : 0.f;
                    sq = fmaf(f[m][c][k], f[m][c][k], sq);
                }
        const float s = rsqrtf(fmaf(group_sum<L>(sq, nullptr), inv, eps));
        if (n >= sh.rows) continue;
        if (lane == 0) stats[n * sh.n_blocks + b] = make_float2(mu, s);
#pragma unroll
        for (int c = 0; c < CG; ++c) {
            if (!at.has_channel(c)) continue;
            float ws[VEC], bs[VEC];
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                ws[k] = w ? w[b * mul + at.channel(c) + k] : 1.f;
                bs[k] = M == 1 && centred && bias ? bias[sh.scalar[b] * mul + at.channel(c) + k] : 0.f;
            }
#pragma unroll
            for (int m = 0; m < P::kRows; ++m) {
#pragma unroll
                for (int k = 0; k < VEC; ++k)
                    f[m][c][k] = M == 1 ? fmaf(f[m][c][k] * s, ws[k], bs[k]) : f[m][c][k] * s * ws[k];
                if (!P::kAlong || at.in(m, c)) store(ys + at.entry(m, c), f[m][c]);
            }
        }
    }
}

template <class TX, class TY, int VEC, int L, int MV, int CG, int U, bool AHEAD, bool KEEP>
__device__ __forceinline__ void irreps_forward(const NormShape& sh, const TX* x, const float* w, const float* bias,
                                               float eps, TY* y, float2* stats) {
    const BlockLanes<L> at;
    for (int64_t n0 = int64_t(blockIdx.x) * at.kPerBlock * U; n0 < sh.rows; n0 += at.step * U) {
        const int64_t n = n0 + threadIdx.x / L;
        if (AHEAD && n + at.step < sh.rows) {   // the node after this one to the L2 cache
            const char* next = reinterpret_cast<const char*>(x + (n + at.step) * sh.x_stride);
            for (int64_t i = at.lane * 128; i < sh.x_stride * int64_t(sizeof(TX)); i += L * 128)
                asm volatile("prefetch.global.L2 [%0];" ::"l"(next + i));
        }
        for (int b = 0; b < sh.n_blocks; ++b) {
            switch (sh.block_rows[b]) {
                case 1: block_forward<TX, TY, VEC, L, MV, CG, 1, U, KEEP>(sh, b, n, at.lane, x, w, bias, eps, y, stats); break;
                case 3: block_forward<TX, TY, VEC, L, MV, CG, 3, U, KEEP>(sh, b, n, at.lane, x, w, bias, eps, y, stats); break;
                case 5: block_forward<TX, TY, VEC, L, MV, CG, 5, U, KEEP>(sh, b, n, at.lane, x, w, bias, eps, y, stats); break;
                default: block_forward<TX, TY, VEC, L, MV, CG, 7, U, KEEP>(sh, b, n, at.lane, x, w, bias, eps, y, stats); break;
            }
        }
    }
}

// bf16 in and out in vectors has half the bytes in flight, and gets more of them by two means (the
// figures: without, with): with 16 and 32 lanes a row two nodes at a time, whose registers allow four
// thread blocks (64,000 x 9 x 128: 60, 50 us; 100,000 x 9 x 64: 50, 44 us), with 4 and 8 lanes the
// next node by a prefetch (200,000 x 9 x 32: 52, 47 us; 500,000 x 9 x 16: 71, 58 us). In fp32 the
// prefetch costs 2-15%, two nodes at a time change nothing or cost up to 7%.
template <class TX, class TY, int VEC, int L, int MV, int CG>
constexpr bool kHalfBytes = sizeof(TX) == 2 && sizeof(TY) == 2 && VEC > 1 && CG == 1 && MV == L && L >= 4;
template <class TX, class TY, int VEC, int L, int MV, int CG>
constexpr bool kPairs = kHalfBytes<TX, TY, VEC, L, MV, CG> && L >= 16;

template <class TX, class TY, int VEC, int L, int MV, int CG, bool KEEP>
__global__ void __launch_bounds__(256)
    irreps_forward_kernel(const __grid_constant__ NormShape sh, const TX* __restrict__ x, const float* __restrict__ w,
                          const float* __restrict__ bias, float eps, TY* __restrict__ y, float2* __restrict__ stats) {
    irreps_forward<TX, TY, VEC, L, MV, CG, 1, kHalfBytes<TX, TY, VEC, L, MV, CG>, KEEP>(sh, x, w, bias, eps, y, stats);
}

template <class TX, class TY, int VEC, int L, int MV, int CG>
__global__ void __launch_bounds__(256, 4)
    irreps_forward_pairs_kernel(const __grid_constant__ NormShape sh, const TX* __restrict__ x,
                                const float* __restrict__ w, const float* __restrict__ bias, float eps,
                                TY* __restrict__ y, float2* __restrict__ stats) {
    irreps_forward<TX, TY, VEC, L, MV, CG, 2, false, true>(sh, x, w, bias, eps, y, stats);
}

// Adds the threads' sums, [block's dw, then even scalar's db][CG][VEC][256], of which every `width`-th
// thread has the same channels, in that order, to out [dw, db][block][mul].
template <int VEC, int L, int CG>
__device__ __forceinline__ void add_lanes(const NormShape& sh, const float* smem, int width, int scalars, float* out) {
    const int mul = int(sh.mul), all = sh.n_blocks * mul, total = all + scalars * mul;
    // few channels: P neighbouring threads add the lanes of one
    int P = 1;
    while (P < 32 && total * P * 2 <= 256 && P * 2 * width <= 256) P *= 2;
    for (int first = 0; first < total; first += 256 / P) {
        const int i = first + int(threadIdx.x) / P, slot = i / mul, q = i - slot * mul, v = q / VEC;
        float a = 0.f;
        if (i < total) {
            const float* from = smem + ((slot * CG + v / L) * VEC + q % VEC) * 256 + v % width;
#pragma unroll 4
            for (int t = (threadIdx.x % P) * width; t < 256; t += P * width) a += from[t];
        }
        for (int o = P / 2; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
        if (i >= total || threadIdx.x % P != 0) continue;
        int to = i;
        if (i >= all)
            for (int b = 0; b < sh.n_blocks; ++b)
                if (sh.scalar[b] == slot - sh.n_blocks) to = all + b * mul + q;
        out[to] = a;
    }
}

// block b of nodes first to last, U nodes a lane at a time; its sums are added to the thread's in smem
template <class TX, class TD, class TO, int VEC, int L, int MV, int CG, int M, int U, bool KEEP>
__device__ __forceinline__ void block_backward(const NormShape& sh, int b, int64_t first, int64_t last, const TX* x,
                                               const float* w, const float2* stats, const TD* dy, TO* dx,
                                               bool sums, float* smem) {
    using P = Place<VEC, L, MV, CG, M>;
    constexpr int kPerBlock = 256 / L;
    const int mul = int(sh.mul);
    const P at(threadIdx.x % L, mul);
    const bool centred = M == 1 && sh.scalar[b] >= 0;
    const float inv = 1.f / float(M * mul);
    const int row0 = sh.first_row[b] * mul + at.first();
    float wv[CG][VEC], dw[CG][VEC], db[CG][VEC];
#pragma unroll
    for (int c = 0; c < CG; ++c)
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
            wv[c][k] = at.has_channel(c) ? (w ? w[b * mul + at.channel(c) + k] : 1.f) : 0.f;
            dw[c][k] = db[c][k] = 0.f;
        }
#pragma unroll 1
    for (int64_t n0 = first; n0 < last; n0 += kPerBlock * U) {
        RawT<TX, VEC> rx[U][P::kRows][CG];
        RawT<TD, VEC> rd[U][P::kRows][CG];
        float2 st[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t n = n0 + threadIdx.x / L + u * kPerBlock;
            const int64_t off = n * sh.x_stride + row0;
            const TX* xs = x + off;
            const TD* ds = dy + off;
            st[u] = n < last ? stats[n * sh.n_blocks + b] : make_float2(0.f, 0.f);
#pragma unroll
            for (int m = 0; m < P::kRows; ++m)
#pragma unroll
                for (int c = 0; c < CG; ++c) {
                    const bool ok = n < last && at.in(m, c);
                    rx[u][m][c] = load_raw<TX, VEC, KEEP>(xs + at.entry(m, c), ok);
                    rd[u][m][c] = load_raw<TD, VEC, KEEP>(ds + at.entry(m, c), ok);
                }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t n = n0 + threadIdx.x / L + u * kPerBlock;
            TO* os = dx + (n * sh.x_stride + row0);
            const float mu = st[u].x, s = st[u].y;
            float xh[P::kRows][CG][VEC], g[P::kRows][CG][VEC], c1 = 0.f, c2 = 0.f;
#pragma unroll
            for (int m = 0; m < P::kRows; ++m)
#pragma unroll
                for (int c = 0; c < CG; ++c) {
                    unpack(rx[u][m][c], xh[m][c]);
                    unpack(rd[u][m][c], g[m][c]);
#pragma unroll
                    for (int k = 0; k < VEC; ++k) {
                        xh[m][c][k] = M == 1 ? (at.in(m, c) ? (xh[m][c][k] - mu) * s : 0.f) : xh[m][c][k] * s;
                        dw[c][k] = fmaf(g[m][c][k], xh[m][c][k], dw[c][k]);
                        if (M == 1) db[c][k] += g[m][c][k];
                        g[m][c][k] *= wv[c][k];
                        if (M == 1) c1 += g[m][c][k];
                        c2 = fmaf(g[m][c][k], xh[m][c][k], c2);
                    }
                }
            // dx = s g - [s mean(g)] - xh s mean(g xh)
            c1 = centred ? -s * (group_sum<L>(c1, nullptr) * inv) : 0.f;
            c2 = -s * (group_sum<L>(c2, nullptr) * inv);
            if (n < last) {
#pragma unroll
                for (int m = 0; m < P::kRows; ++m)
#pragma unroll
                    for (int c = 0; c < CG; ++c) {
#pragma unroll
                        for (int k = 0; k < VEC; ++k)
                            g[m][c][k] = fmaf(xh[m][c][k], c2, M == 1 ? fmaf(g[m][c][k], s, c1) : g[m][c][k] * s);
                        if (at.in(m, c)) store(os + at.entry(m, c), g[m][c]);
                    }
            }
        }
    }
    if (!sums) return;
    float* own = smem + b * (CG * VEC * 256) + threadIdx.x;
#pragma unroll
    for (int c = 0; c < CG; ++c)
#pragma unroll
        for (int k = 0; k < VEC; ++k) own[(c * VEC + k) * 256] += dw[c][k];
    if (!centred) return;
    own = smem + (sh.n_blocks + sh.scalar[b]) * (CG * VEC * 256) + threadIdx.x;
#pragma unroll
    for (int c = 0; c < CG; ++c)
#pragma unroll
        for (int k = 0; k < VEC; ++k) own[(c * VEC + k) * 256] += db[c][k];
}

// Shared memory: a thread's sums, [block's dw, then even scalar's db][CG][VEC][256].
template <class TX, class TD, class TO, int VEC, int L, int MV, int CG, bool KEEP>
__global__ void __launch_bounds__(256, VEC == 4 ? (CG == 1 ? 3 : 1) : CG <= 2 ? 5 : CG == 4 ? 2 : 1)
    irreps_backward_kernel(const __grid_constant__ NormShape sh, const TX* __restrict__ x, const float* __restrict__ w,
                           const float2* __restrict__ stats, const TD* __restrict__ dy, TO* __restrict__ dx,
                           float* __restrict__ partial, int64_t tile) {
    asm volatile("griddepcontrol.launch_dependents;");
    extern __shared__ float smem[];
    const bool sums = partial != nullptr;
    int scalars = 0;
    for (int b = 0; b < sh.n_blocks; ++b) scalars += sh.scalar[b] >= 0;
    if (sums)
        for (int i = 0; i < (sh.n_blocks + scalars) * (CG * VEC); ++i) smem[i * 256 + threadIdx.x] = 0.f;
    // few vectors in a segment: several nodes at a time keep as many loads in flight
    constexpr bool kAlong = MV < L;
    constexpr int U1 = VEC == 1 ? (CG <= 2 ? 4 / CG : 1) : CG > 1 ? 1 : kAlong ? 4 : 2;
    constexpr int U3 = CG > 1 ? 1 : kAlong ? 4 : 2, U5 = kAlong ? 2 : 1;
    for (int64_t first = blockIdx.x * tile; first < sh.rows; first += gridDim.x * tile) {
        const int64_t last = first + tile < sh.rows ? first + tile : sh.rows;
        for (int b = 0; b < sh.n_blocks; ++b) {
            switch (sh.block_rows[b]) {
                case 1: block_backward<TX, TD, TO, VEC, L, MV, CG, 1, U1, KEEP>(sh, b, first, last, x, w, stats, dy, dx, sums, smem); break;
                case 3: block_backward<TX, TD, TO, VEC, L, MV, CG, 3, U3, KEEP>(sh, b, first, last, x, w, stats, dy, dx, sums, smem); break;
                case 5: block_backward<TX, TD, TO, VEC, L, MV, CG, 5, U5, KEEP>(sh, b, first, last, x, w, stats, dy, dx, sums, smem); break;
                default: block_backward<TX, TD, TO, VEC, L, MV, CG, 7, U5, KEEP>(sh, b, first, last, x, w, stats, dy, dx, sums, smem); break;
            }
        }
    }
    if (!sums) return;
    __syncthreads();
    add_lanes<VEC, L, CG>(sh, smem, MV < L ? int(sh.mul) / VEC : L, scalars,
                          partial + int64_t(blockIdx.x) * 2 * sh.n_blocks * sh.mul);
}

}  // namespace blocks
}  // namespace e3gb
