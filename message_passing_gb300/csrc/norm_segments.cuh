// Layer norm in registers: L lanes (a part of a warp, a warp, or a block) own a row and hold it in
// vectors of VEC entries, lane k the vectors k, k + L, ... (NV of them).
//
// Bound by memory: every entry is read once and written once. A thread's next rows arrive in shared
// memory (each thread copies what it will read itself, so that no barrier is needed) while it works
// on one; mean, variance and output come from the registers. A lane's channels are the same in every
// row that it takes, so that it sums its part of dw and db over all of them; one partial sum per
// thread block goes to memory. Measured, of the copy rate: forward 2.56M x 64 bf16 107 us (93%),
// backward 131,072 x 1024 bf16 127 us (94%), 1M x 128 fp32 162 us (93%) and 236 us (96%).
//
// Rows that are not whole vectors (ODD): a row's first entry then lies `shift` entries into a vector,
// and shift depends on the row modulo VEC only. A lane group's rows are a multiple of VEC apart, so
// that its channels still are the same in all of them; the vectors at the two ends hold entries of
// the rows beside, which are masked, and are written entry by entry. Rows of more than about 70
// entries reach 70-95% of the copy rate in fp32 (50,021 x 321, backward: 36 us, 78%; 701 columns 53%); in bf16, and
// narrower, the masks and the lanes past the end make the instructions the bound (39-60%).
#pragma once
#include "async_copy.cuh"
#include "norm.cuh"

namespace e3gb {
namespace segments {

using bf16 = __nv_bfloat16;

// ------------------------------------------------------------------------------------------
// vectors of VEC neighbouring entries, raw and in fp32
// ------------------------------------------------------------------------------------------
template <class T, int VEC>
struct Raw;
template <>
struct Raw<float, 1> { using type = float; };
template <>
struct Raw<bf16, 1> { using type = unsigned short; };
template <>
struct Raw<float, 4> { using type = float4; };
template <>
struct Raw<bf16, 4> { using type = uint2; };
template <>
struct Raw<bf16, 8> { using type = uint4; };
template <class T, int VEC>
using RawT = typename Raw<T, VEC>::type;

__device__ __forceinline__ float lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float hi(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }
__device__ __forceinline__ void unpack(float r, float (&f)[1]) { f[0] = r; }
__device__ __forceinline__ void unpack(unsigned short r, float (&f)[1]) { f[0] = lo(r); }
__device__ __forceinline__ void unpack(const float4& r, float (&f)[4]) { f[0] = r.x, f[1] = r.y, f[2] = r.z, f[3] = r.w; }
__device__ __forceinline__ void unpack(const uint2& r, float (&f)[4]) { f[0] = lo(r.x), f[1] = hi(r.x), f[2] = lo(r.y), f[3] = hi(r.y); }
__device__ __forceinline__ void unpack(const uint4& r, float (&f)[8]) {
    f[0] = lo(r.x), f[1] = hi(r.x), f[2] = lo(r.y), f[3] = hi(r.y);
    f[4] = lo(r.z), f[5] = hi(r.z), f[6] = lo(r.w), f[7] = hi(r.w);
}
__device__ __forceinline__ uint32_t pair(float a, float b) {
    const __nv_bfloat162 t = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&t);
}
__device__ __forceinline__ void store(float* p, const float (&f)[1]) { *p = f[0]; }
__device__ __forceinline__ void store(bf16* p, const float (&f)[1]) { *p = __float2bfloat16_rn(f[0]); }
__device__ __forceinline__ void store(float* p, const float (&f)[4]) { *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]); }
__device__ __forceinline__ void store(bf16* p, const float (&f)[4]) { *reinterpret_cast<uint2*>(p) = make_uint2(pair(f[0], f[1]), pair(f[2], f[3])); }
__device__ __forceinline__ void store(bf16* p, const float (&f)[8]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pair(f[0], f[1]), pair(f[2], f[3]), pair(f[4], f[5]), pair(f[6], f[7]));
}
__device__ __forceinline__ void store_one(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_one(bf16* p, float v) { *p = __float2bfloat16_rn(v); }

// ------------------------------------------------------------------------------------------
// sums
// ------------------------------------------------------------------------------------------
// over the L lanes that share a segment; L > 32: over the block, through smem (N arrays of L / 32 floats),
// with one barrier. smem must not be the one that was read after the barrier before.
template <int L, int N>
__device__ __forceinline__ void group_sums(float (&v)[N], float* smem) {
#pragma unroll
    for (int o = (L < 32 ? L : 32) / 2; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    if constexpr (L > 32) {
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) smem[i * (L / 32) + (threadIdx.x >> 5)] = v[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            v[i] = smem[i * (L / 32)];
#pragma unroll
            for (int k = 1; k < L / 32; ++k) v[i] += smem[i * (L / 32) + k];
        }
    }
}
template <int L>
__device__ __forceinline__ float group_sum(float v, float* smem) {
    float a[1] = {v};
    group_sums<L>(a, smem);
    return a[0];
}

// ------------------------------------------------------------------------------------------
// rows of a thread
// ------------------------------------------------------------------------------------------
template <int L>
constexpr int kThreads = L > 32 ? L : 256;

// A thread's rows: `first`, then every `step`-th, `mine` in all. The threads of a block go round `turns`
// times together, since they reduce together. ODD: step is a multiple of VEC (the lane groups of a
// block are, or the grid is).
template <int L>
struct Lanes {
    static constexpr int kPerBlock = kThreads<L> / L;   // rows that a block takes at a time
    int lane;   // among the L
    int64_t first, step;
    int mine, turns;
    __device__ __forceinline__ explicit Lanes(int64_t rows) {
        lane = threadIdx.x % L;
        const int64_t start = int64_t(blockIdx.x) * kPerBlock;
        first = start + int64_t(threadIdx.x / L);
        step = int64_t(gridDim.x) * kPerBlock;
        mine = first < rows ? int((rows - 1 - first) / step) + 1 : 0;
        turns = start < rows ? int((rows - 1 - start) / step) + 1 : 0;
    }
};

// rows `stride` entries apart; all of them end at `end`
template <class T>
struct Tensor {
    T* at;
    int64_t stride;
    const T* end;
};

// how a row's entries lie in a lane's vectors: entry (j, k) is number (lane + j L) VEC + k - shift
template <int VEC, int L, int NV, bool ODD>
struct Layout {
    int lane, vecs, K, shift;
    __device__ __forceinline__ int entry(int j, int k) const { return (lane + j * L) * VEC + k - (ODD ? shift : 0); }
    __device__ __forceinline__ bool has(int j, int k) const {
        return ODD ? unsigned(entry(j, k)) < unsigned(K) : lane + j * L < vecs;
    }
    __device__ __forceinline__ bool any(int j) const { return lane + j * L < vecs; }
    __device__ __forceinline__ bool all(int j) const {
        if (!ODD) return any(j);
        return entry(j, 0) >= 0 && entry(j, VEC - 1) < K;
    }
    template <class T>
    __device__ __forceinline__ static Layout of(const T* row, int lane, int K) {
        Layout y;
        y.lane = lane;
        y.K = K;
        y.shift = ODD ? int((reinterpret_cast<uintptr_t>(row) / sizeof(T)) % VEC) : 0;
        y.vecs = (K + y.shift + VEC - 1) / VEC;
        return y;
    }
};

// rows of every thread in shared memory
template <class T, int VEC, int L, int NV, bool ODD>
struct Ring {
    static constexpr int THREADS = kThreads<L>;
    using R = RawT<T, VEC>;
    static constexpr int kBytes = int(sizeof(R)) * NV * THREADS;

    // row: its first entry. Vectors past the last one read as zero: their copies read nothing, but have a source
    // address all the same, which has to be aligned. A tensor of ODD rows may begin inside a vector; that
    // vector's start is in the same 16 bytes of memory as the tensor's.
    static __device__ __forceinline__ void fetch(char* slot, const Tensor<T>& t, const T* row,
                                                 const Layout<VEC, L, NV, ODD>& y, bool live) {
        const T* nothing = ODD ? reinterpret_cast<const T*>(reinterpret_cast<uintptr_t>(t.at) & ~uintptr_t(sizeof(R) - 1)) : t.at;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            R* to = reinterpret_cast<R*>(slot) + j * THREADS + threadIdx.x;
            const bool ok = live && y.any(j);
            const T* from = row + y.entry(j, 0);
            if constexpr (ODD) {
                if (ok && (from < t.at || from + VEC > t.end)) {   // the tensor begins or ends inside this vector
                    for (int k = 0; k < VEC; ++k)
                        if (y.has(j, k)) reinterpret_cast<T*>(to)[k] = from[k];
                    continue;
                }
            }
            copy_async<sizeof(R)>(to, ok ? from : nothing, ok);
        }
    }
    static __device__ __forceinline__ R get(const char* slot, int j) {
        return reinterpret_cast<const R*>(slot)[j * THREADS + threadIdx.x];
    }
};

template <int VEC, int L, int NV, bool ODD>
__device__ __forceinline__ void mask(float (&f)[VEC], const Layout<VEC, L, NV, ODD>& y, int j) {
    if (ODD && !y.all(j))
#pragma unroll
        for (int k = 0; k < VEC; ++k) f[k] = y.has(j, k) ? f[k] : 0.f;
}
template <class T, int VEC, int L, int NV, bool ODD>
__device__ __forceinline__ void put(T* row, const float (&f)[VEC], const Layout<VEC, L, NV, ODD>& y, int j) {
    if (y.all(j)) {
        store(row + y.entry(j, 0), f);
    } else if (ODD && y.any(j)) {
#pragma unroll
        for (int k = 0; k < VEC; ++k)
            if (y.has(j, k)) store_one(row + y.entry(j, k), f[k]);
    }
}

template <class TX, class TY, int VEC, int L, int NV, int S, bool ODD>
__global__ void __launch_bounds__(kThreads<L>, L > 32 || NV * VEC > 16 ? 1 : NV * VEC <= 8 ? 4 : 2)
    forward_kernel(int64_t rows, int cols, Tensor<TX> x, Tensor<TY> y, const float* __restrict__ w,
                   const float* __restrict__ bias, float eps, float2* __restrict__ stats) {
    using X = Ring<TX, VEC, L, NV, ODD>;
    extern __shared__ __align__(16) char ring[];
    __shared__ float smem[2][kThreads<L> / 32];
    const Lanes<L> at(rows);
    const int64_t from = at.mine > 0 ? at.first : 0;
    TX* ahead = x.at + from * x.stride;
    const auto lay = Layout<VEC, L, NV, ODD>::of(ahead, at.lane, cols);
    const float inv = 1.f / float(cols);
    float wv[NV][VEC], bv[NV][VEC];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
            const bool in = lay.has(j, k);
            wv[j][k] = in ? (w ? w[lay.entry(j, k)] : 1.f) : 0.f;
            bv[j][k] = in && bias ? bias[lay.entry(j, k)] : 0.f;
        }
    const int64_t x_step = at.step * x.stride, y_step = at.step * y.stride;
    int put_at = 0, get_at = 0;
    const auto fetch = [&](int i) {
        X::fetch(ring + put_at * X::kBytes, x, ahead, lay, i < at.mine);
        copies_commit();
        ahead += x_step;
        put_at = put_at + 1 == S ? 0 : put_at + 1;
    };
#pragma unroll
    for (int i = 0; i < S - 1; ++i) fetch(i);
    TY* ys = y.at + from * y.stride;
    float2* st = stats + from;
#pragma unroll 1
    for (int i = 0; i < at.turns; ++i) {
        fetch(i + S - 1);
        copies_wait<S - 1>();
        float f[NV][VEC], sum = 0.f, sq = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            unpack(X::get(ring + get_at * X::kBytes, j), f[j]);
            mask(f[j], lay, j);
#pragma unroll
            for (int k = 0; k < VEC; ++k) sum += f[j][k];   // entries outside are zero
        }
        get_at = get_at + 1 == S ? 0 : get_at + 1;
        const float mu = group_sum<L>(sum, smem[0]) * inv;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
#pragma unroll
            for (int k = 0; k < VEC; ++k) f[j][k] -= mu;
            if constexpr (ODD) {
                mask(f[j], lay, j);
            } else {
                if (!lay.any(j))
#pragma unroll
                    for (int k = 0; k < VEC; ++k) f[j][k] = 0.f;
            }
#pragma unroll
            for (int k = 0; k < VEC; ++k) sq = fmaf(f[j][k], f[j][k], sq);
        }
        const float s = rsqrtf(fmaf(group_sum<L>(sq, smem[1]), inv, eps));
        if (i < at.mine) {
            if (at.lane == 0) *st = make_float2(mu, s);
#pragma unroll
            for (int j = 0; j < NV; ++j) {
#pragma unroll
                for (int k = 0; k < VEC; ++k) f[j][k] = fmaf(f[j][k] * s, wv[j][k], bv[j][k]);
                put(ys, f[j], lay, j);
            }
        }
        ys += y_step;
        st += at.step;
    }
    copies_wait<0>();
}

// partial [gridDim.x][2][cols]: this block's sums of dy xh and of dy (or null)
template <class TX, class TD, class TO, int VEC, int L, int NV, int S, bool ODD>
__global__ void __launch_bounds__(kThreads<L>, L > 32 || NV * VEC > 16 ? 1 : NV * VEC <= 4 ? 4 : NV * VEC <= 8 ? 3 : 2)
    backward_kernel(int64_t rows, int cols, Tensor<TX> x, Tensor<TD> dy, Tensor<TO> dx, const float* __restrict__ w,
                    const float2* __restrict__ stats, float* __restrict__ partial) {
    using X = Ring<TX, VEC, L, NV, ODD>;
    using D = Ring<TD, VEC, L, NV, ODD>;
    constexpr int T = kThreads<L>, kSlot = X::kBytes + D::kBytes + 8 * T;
    // with many entries a lane, xh and g are formed again from shared memory instead of being held
    constexpr bool kAgain = NV * VEC > 16;
    extern __shared__ __align__(16) char ring[];
    __shared__ float smem[L > 32 ? 4 * (L / 32) : 1];
    asm volatile("griddepcontrol.launch_dependents;");
    const Lanes<L> at(rows);
    const int64_t from = at.mine > 0 ? at.first : 0;
    TX* x_ahead = x.at + from * x.stride;
    TD* dy_ahead = dy.at + from * dy.stride;
    const float2* st_ahead = stats + from;
    const auto lay = Layout<VEC, L, NV, ODD>::of(x_ahead, at.lane, cols);
    const float inv = 1.f / float(cols);
    float wv[NV][VEC], dw[NV][VEC], db[NV][VEC];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
            wv[j][k] = lay.has(j, k) ? (w ? w[lay.entry(j, k)] : 1.f) : 0.f;
            dw[j][k] = db[j][k] = 0.f;
        }
    const int64_t x_step = at.step * x.stride, dy_step = at.step * dy.stride, dx_step = at.step * dx.stride;
    int put_at = 0, get_at = 0;
    const auto fetch = [&](int i) {
        char* slot = ring + put_at * kSlot;
        const bool live = i < at.mine;
        X::fetch(slot, x, x_ahead, lay, live);
        D::fetch(slot + X::kBytes, dy, dy_ahead, lay, live);
        copy_async<8>(reinterpret_cast<float2*>(slot + X::kBytes + D::kBytes) + threadIdx.x, live ? st_ahead : stats, live);
        copies_commit();
        x_ahead += x_step;
        dy_ahead += dy_step;
        st_ahead += at.step;
        put_at = put_at + 1 == S ? 0 : put_at + 1;
    };
#pragma unroll
    for (int i = 0; i < S - 1; ++i) fetch(i);
    TO* os = dx.at + from * dx.stride;
#pragma unroll 1
    for (int i = 0; i < at.turns; ++i) {
        fetch(i + S - 1);
        copies_wait<S - 1>();
        const char* slot = ring + get_at * kSlot;
        const float2 st = reinterpret_cast<const float2*>(slot + X::kBytes + D::kBytes)[threadIdx.x];
        const float mu = st.x, s = st.y;
        float xh[kAgain ? 1 : NV][VEC], g[kAgain ? 1 : NV][VEC], c[2] = {0.f, 0.f};
        const auto form = [&](int j, float (&xv)[VEC], float (&gv)[VEC]) {   // xh and dy of vector j
            unpack(X::get(slot, j), xv);
            unpack(D::get(slot + X::kBytes, j), gv);
#pragma unroll
            for (int k = 0; k < VEC; ++k) xv[k] = (xv[k] - mu) * s;   // x s - mu s would round mu s, of a large mean
            mask(xv, lay, j);
            mask(gv, lay, j);
            if (!ODD && !lay.any(j))
#pragma unroll
                for (int k = 0; k < VEC; ++k) xv[k] = 0.f;
        };
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            float (&xv)[VEC] = xh[kAgain ? 0 : j], (&gv)[VEC] = g[kAgain ? 0 : j];
            form(j, xv, gv);
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                dw[j][k] = fmaf(gv[k], xv[k], dw[j][k]);
                db[j][k] += gv[k];
                gv[k] *= wv[j][k];
                c[0] += gv[k];
                c[1] = fmaf(gv[k], xv[k], c[1]);
            }
        }
        group_sums<L>(c, smem + (i & 1) * 2 * (L / 32));
        // dx = s g - s mean(g) - xh s mean(g xh)
        const float c1 = -s * (c[0] * inv), c2 = -s * (c[1] * inv);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            float (&xv)[VEC] = xh[kAgain ? 0 : j], (&gv)[VEC] = g[kAgain ? 0 : j];
            if constexpr (kAgain) {
                form(j, xv, gv);
#pragma unroll
                for (int k = 0; k < VEC; ++k) gv[k] *= wv[j][k];
            }
#pragma unroll
            for (int k = 0; k < VEC; ++k) gv[k] = fmaf(xv[k], c2, fmaf(gv[k], s, c1));
            if (i < at.mine) put(os, gv, lay, j);
        }
        get_at = get_at + 1 == S ? 0 : get_at + 1;
        os += dx_step;
    }
    copies_wait<0>();
    if (partial == nullptr) return;
    __syncthreads();
    float* out = partial + int64_t(blockIdx.x) * 2 * cols;
    // by channels (the lane groups of ODD rows are shifted differently), over the lane groups in their order
    float* by_group = reinterpret_cast<float*>(ring);   // [T / L][cols]
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        float* to = L < T ? by_group + int(threadIdx.x / L) * cols : out + which * cols;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int k = 0; k < VEC; ++k)
                if (lay.has(j, k)) to[lay.entry(j, k)] = which ? db[j][k] : dw[j][k];
        if constexpr (L < T) {
            __syncthreads();
            for (int c = threadIdx.x; c < cols; c += T) {
                float a = 0.f;
#pragma unroll 8
                for (int i = 0; i < T / L; ++i) a += by_group[i * cols + c];
                out[which * cols + c] = a;
            }
            __syncthreads();
        }
    }
}

}  // namespace segments
}  // namespace e3gb
