// Layer norm of rows whose tensors are aligned differently (a strided odd-width input with a contiguous
// output, say), so that no vector of one lies over a vector of another.
//
// A group of threads (a warp, or a block for long rows) takes tiles of T neighbouring rows. A tile is
// copied to shared memory 16 bytes at a time, whatever the rows' length and alignment: rows that are
// whole 16-byte units one by one, each to a padded place, so that rows read side by side lie in
// different banks; others as the one span of units that covers them. Entries are then read one by
// one, lane by channel, and the results go back through shared memory the same way. Bound by the
// instructions that this takes: 45-65% of the copy rate in fp32 and 21-35% in bf16.
#pragma once
#include "async_copy.cuh"
#include "norm.cuh"

namespace e3gb {
namespace flat {

using bf16 = __nv_bfloat16;

// one tensor of rows, by bytes
struct Rows {
    char* base;
    char* end;            // one past the last row's last byte
    int64_t stride;
    int row;              // bytes of a row
    int pitch;            // between rows in shared memory
    int slot;             // bytes of a tile in shared memory
    bool units;           // every row is whole 16-byte units
};

// where a tile lies in shared memory
struct Place {
    char* at;             // of the first row
    int pitch;
};

template <int GROUP>
__device__ __forceinline__ void group_sync() {
    if constexpr (GROUP == 32) __syncwarp();
    else __syncthreads();
}

__device__ __forceinline__ Place place(const Rows& r, char* slot, int64_t row) {
    if (r.units) return {slot, r.pitch};
    return {slot + (reinterpret_cast<uintptr_t>(r.base + row * r.stride) & 15), r.pitch};
}

// Walks the 16-byte units of rows [row, row + n): f(unit in memory, unit in shared memory). `lane` of
// GROUP threads takes every GROUP-th.
template <int GROUP, class F>
__device__ __forceinline__ void units(const Rows& r, char* slot, int64_t row, int n, int lane, F&& f) {
    char* start = r.base + row * r.stride;
    if (r.units) {
        const int per = r.row / 16, dt = GROUP / per, dc = GROUP % per;
        int t = lane / per, c = lane % per;
        while (t < n) {
            f(start + t * r.stride + c * 16, slot + t * r.pitch + c * 16);
            t += dt;
            c += dc;
            if (c >= per) c -= per, ++t;
        }
    } else {
        const int shift = int(reinterpret_cast<uintptr_t>(start) & 15);
        const int bytes = shift + (n - 1) * r.pitch + r.row;   // n > 1: the rows follow one another
        for (int u = lane * 16; u < bytes; u += GROUP * 16) f(start - shift + u, slot + u);
    }
}

template <class T, int GROUP>
__device__ __forceinline__ void fetch(const Rows& r, char* slot, int64_t row, int n, int lane) {
    units<GROUP>(r, slot, row, n, lane, [&](char* from, char* to) {
        if (from >= r.base && from + 16 <= r.end) {
            copy_async<16>(to, from);
        } else {   // the tensor's first or last unit, which it fills in part
            for (int k = 0; k < 16; k += int(sizeof(T)))
                if (from + k >= r.base && from + k < r.end) *reinterpret_cast<T*>(to + k) = *reinterpret_cast<const T*>(from + k);
        }
    });
}

template <class T, int GROUP>
__device__ __forceinline__ void put_back(const Rows& r, char* slot, int64_t row, int n, int lane) {
    const char* first = r.base + row * r.stride;
    const char* last = first + (n - 1) * r.stride + r.row;
    units<GROUP>(r, slot, row, n, lane, [&](char* to, char* from) {
        if (to >= first && to + 16 <= last) {
            *reinterpret_cast<uint4*>(to) = *reinterpret_cast<const uint4*>(from);
        } else {
            for (int k = 0; k < 16; k += int(sizeof(T)))
                if (to + k >= first && to + k < last) *reinterpret_cast<T*>(to + k) = *reinterpret_cast<const T*>(from + k);
        }
    });
}

__device__ __forceinline__ float get(const float* p) { return *p; }
__device__ __forceinline__ float get(const bf16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void set(float* p, float v) { *p = v; }
__device__ __forceinline__ void set(bf16* p, float v) { *p = __float2bfloat16_rn(v); }

// lanes: L for a segment (all of a longer group), G segments of a group side by side
template <int L, int GROUP>
struct Threads {
    static constexpr int G = GROUP / L;
    int lane, sub, l, group;
    __device__ __forceinline__ Threads()
        : lane(threadIdx.x % GROUP), sub(lane / L), l(lane % L), group(threadIdx.x / GROUP) {}
};

template <int GROUP, int L, int N>
__device__ __forceinline__ void sums(float (&v)[N], float* smem) {
#pragma unroll
    for (int o = (L < 32 ? L : 32) / 2; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    if constexpr (GROUP > 32) {
        __syncthreads();   // the sums before these have been read
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) smem[i * (GROUP / 32) + (threadIdx.x >> 5)] = v[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            v[i] = 0.f;
#pragma unroll
            for (int k = 0; k < GROUP / 32; ++k) v[i] += smem[i * (GROUP / 32) + k];
        }
    }
}

// rows that a lane has in hand at once: few entries each, so that their sums' latencies overlap
template <int ENTRIES, int GROUP>
constexpr int kSide = GROUP > 32 || ENTRIES > 4 ? 1 : ENTRIES > 2 ? 2 : 4;

// the n rows of a tile, CG channels a lane
template <class TX, class TY, int L, int CG, int GROUP>
__device__ __forceinline__ void forward_tile(int mul, int n, Place x, Place y, const float (&wv)[CG], const float (&bv)[CG],
                                             float eps, float2* stats, float* smem) {
    constexpr int U = kSide<CG, GROUP>;
    const Threads<L, GROUP> th;
    const float inv = 1.f / float(mul);
    const TX* x0 = reinterpret_cast<const TX*>(x.at) + th.l;
    TY* y0 = reinterpret_cast<TY*>(y.at) + th.l;
    const int x_pitch = x.pitch / int(sizeof(TX)), y_pitch = y.pitch / int(sizeof(TY));
    for (int t0 = th.sub; t0 < n + th.sub; t0 += U * th.G) {
        float f[U][CG], a[U], mu[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int t = t0 + u * th.G;
            const TX* xs = x0 + (t < n ? t : 0) * x_pitch;
            a[u] = 0.f;
#pragma unroll
            for (int j = 0; j < CG; ++j) {
                f[u][j] = th.l + j * L < mul ? get(xs + j * L) : 0.f;
                a[u] += f[u][j];
            }
        }
        sums<GROUP, L>(a, smem);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            mu[u] = a[u] * inv;
            a[u] = 0.f;
#pragma unroll
            for (int j = 0; j < CG; ++j) {
                f[u][j] = th.l + j * L < mul ? f[u][j] - mu[u] : 0.f;
                a[u] = fmaf(f[u][j], f[u][j], a[u]);
            }
        }
        sums<GROUP, L>(a, smem);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int t = t0 + u * th.G;
            const float s = rsqrtf(fmaf(a[u], inv, eps));
            if (t >= n) continue;
            if (th.l == 0) stats[t] = make_float2(mu[u], s);
            TY* ys = y0 + t * y_pitch;
#pragma unroll
            for (int j = 0; j < CG; ++j)
                if (th.l + j * L < mul) set(ys + j * L, fmaf(f[u][j] * s, wv[j], bv[j]));
        }
    }
}

// dw, db: this lane's sums
template <class TX, class TD, class TO, int L, int CG, int GROUP>
__device__ __forceinline__ void backward_tile(int mul, int n, Place x, Place d, Place o, const float (&wv)[CG],
                                              const float2* stats, float* smem, float (&dw)[CG], float (&db)[CG]) {
    constexpr bool kAgain = CG > 12;   // xh and g are formed again instead of being held
    constexpr int U = kAgain ? 1 : kSide<CG, GROUP>, HC = kAgain ? 1 : CG;
    const Threads<L, GROUP> th;
    const float inv = 1.f / float(mul);
    const TX* x0 = reinterpret_cast<const TX*>(x.at) + th.l;
    const TD* d0 = reinterpret_cast<const TD*>(d.at) + th.l;
    TO* o0 = reinterpret_cast<TO*>(o.at) + th.l;
    const int x_pitch = x.pitch / int(sizeof(TX)), d_pitch = d.pitch / int(sizeof(TD)), o_pitch = o.pitch / int(sizeof(TO));
    for (int t0 = th.sub; t0 < n + th.sub; t0 += U * th.G) {
        float xh[U][HC], g[U][HC], c[2 * U];
        float2 st[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int t = t0 + u * th.G, tt = t < n ? t : 0;
            const TX* xs = x0 + tt * x_pitch;
            const TD* ds = d0 + tt * d_pitch;
            st[u] = stats[tt];
            c[2 * u] = c[2 * u + 1] = 0.f;
#pragma unroll
            for (int j = 0; j < CG; ++j) {
                const bool in = t < n && th.l + j * L < mul;
                const float xv = in ? (get(xs + j * L) - st[u].x) * st[u].y : 0.f;
                const float dv = in ? get(ds + j * L) : 0.f, gv = dv * wv[j];
                dw[j] = fmaf(dv, xv, dw[j]);
                db[j] += dv;
                c[2 * u + 1] += gv;
                c[2 * u] = fmaf(gv, xv, c[2 * u]);
                if (!kAgain) xh[u][kAgain ? 0 : j] = xv, g[u][kAgain ? 0 : j] = gv;
            }
        }
        sums<GROUP, L>(c, smem);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int t = t0 + u * th.G;
            if (t >= n) continue;
            const float c1 = c[2 * u + 1] * inv, c2 = c[2 * u] * inv, mu = st[u].x, s = st[u].y;
            const TX* xs = x0 + t * x_pitch;
            const TD* ds = d0 + t * d_pitch;
            TO* os = o0 + t * o_pitch;
#pragma unroll
            for (int j = 0; j < CG; ++j) {
                if (th.l + j * L >= mul) continue;
                const float xv = kAgain ? (get(xs + j * L) - mu) * s : xh[u][kAgain ? 0 : j];
                const float gv = kAgain ? get(ds + j * L) * wv[j] : g[u][kAgain ? 0 : j];
                set(os + j * L, s * (gv - c1 - xv * c2));
            }
        }
    }
}

template <int L, int CG>
__device__ __forceinline__ void weights(int mul, int l, const float* w, float none, float (&wv)[CG]) {
#pragma unroll
    for (int j = 0; j < CG; ++j) wv[j] = l + j * L < mul && w ? w[l + j * L] : none;
}

constexpr int kTiles = 3;   // of a group in shared memory: one in hand, the others on their way

// Shared memory of a group: kTiles tiles of x, one of y.
template <class TX, class TY, int L, int CG, int GROUP>
__global__ void __launch_bounds__(GROUP > 32 ? GROUP : 256)
    forward_kernel(const __grid_constant__ NormShape sh, const __grid_constant__ Rows x, const __grid_constant__ Rows y,
                   int tile, const float* __restrict__ w, const float* __restrict__ bias, float eps,
                   float2* __restrict__ stats) {
    extern __shared__ __align__(16) char memory[];
    __shared__ float smem[GROUP > 32 ? GROUP / 32 : 1];
    const Threads<L, GROUP> th;
    char* mine = memory + th.group * (kTiles * x.slot + y.slot);
    char* out = mine + kTiles * x.slot;
    const int64_t groups = int64_t(gridDim.x) * (blockDim.x / GROUP);
    int64_t row = (int64_t(blockIdx.x) * (blockDim.x / GROUP) + th.group) * tile, ahead = row;
    const int64_t step = groups * tile;
    const auto count = [&](int64_t r) { return r >= sh.rows ? 0 : sh.rows - r < tile ? int(sh.rows - r) : tile; };
    int put = 0, now = 0;
    const auto load = [&] {
        const int n = count(ahead);
        if (n > 0) fetch<TX, GROUP>(x, mine + put * x.slot, ahead, n, th.lane);
        copies_commit();
        ahead += step;
        put = put + 1 == kTiles ? 0 : put + 1;
    };
    float wv[CG], bv[CG];
    weights<L>(int(sh.mul), th.l, w, 1.f, wv);
    weights<L>(int(sh.mul), th.l, bias, 0.f, bv);
    for (int i = 0; i < kTiles - 1; ++i) load();
    for (; row < sh.rows; row += step) {
        load();
        copies_wait<kTiles - 1>();
        group_sync<GROUP>();
        const int n = count(row);
        const Place px = place(x, mine + now * x.slot, row), py = place(y, out, row);
        forward_tile<TX, TY, L, CG, GROUP>(int(sh.mul), n, px, py, wv, bv, eps, stats + row, smem);
        group_sync<GROUP>();
        put_back<TY, GROUP>(y, out, row, n, th.lane);
        group_sync<GROUP>();
        now = now + 1 == kTiles ? 0 : now + 1;
    }
    copies_wait<0>();
}

// Shared memory of a group: kTiles tiles of x, dy and stats and one of dx; at the end, in their place, the
// lanes' sums [dw, db][CG][GROUP]. partial [gridDim.x][2][mul].
template <class TX, class TD, class TO, int L, int CG, int GROUP>
__global__ void __launch_bounds__(GROUP > 32 ? GROUP : 256)
    backward_kernel(const __grid_constant__ NormShape sh, const __grid_constant__ Rows x, const __grid_constant__ Rows d,
                    const __grid_constant__ Rows o, int tile, int each, const float* __restrict__ w,
                    const float2* __restrict__ stats, float* __restrict__ partial) {
    extern __shared__ __align__(16) char memory[];
    __shared__ float smem[GROUP > 32 ? 2 * (GROUP / 32) : 1];
    const Threads<L, GROUP> th;
    asm volatile("griddepcontrol.launch_dependents;");
    const int mul = int(sh.mul), slot = x.slot + d.slot + (tile * 8 + 15) / 16 * 16;
    char* mine = memory + th.group * each;
    char* out = mine + kTiles * slot;
    const int64_t groups = int64_t(gridDim.x) * (blockDim.x / GROUP);
    int64_t row = (int64_t(blockIdx.x) * (blockDim.x / GROUP) + th.group) * tile, ahead = row;
    const int64_t step = groups * tile;
    const auto count = [&](int64_t r) { return r >= sh.rows ? 0 : sh.rows - r < tile ? int(sh.rows - r) : tile; };
    int put = 0, now = 0;
    const auto load = [&] {
        const int n = count(ahead);
        char* to = mine + put * slot;
        if (n > 0) {
            fetch<TX, GROUP>(x, to, ahead, n, th.lane);
            fetch<TD, GROUP>(d, to + x.slot, ahead, n, th.lane);
            float2* st = reinterpret_cast<float2*>(to + x.slot + d.slot);
            for (int i = th.lane; i < n; i += GROUP) copy_async<8>(st + i, stats + ahead + i);
        }
        copies_commit();
        ahead += step;
        put = put + 1 == kTiles ? 0 : put + 1;
    };
    float wv[CG], dw[CG], db[CG];
#pragma unroll
    for (int j = 0; j < CG; ++j) dw[j] = db[j] = 0.f;
    weights<L>(mul, th.l, w, 1.f, wv);
    for (int i = 0; i < kTiles - 1; ++i) load();
    for (; row < sh.rows; row += step) {
        load();
        copies_wait<kTiles - 1>();
        group_sync<GROUP>();
        const int n = count(row);
        char* in = mine + now * slot;
        const Place px = place(x, in, row), pd = place(d, in + x.slot, row), po = place(o, out, row);
        const float2* st = reinterpret_cast<const float2*>(in + x.slot + d.slot);
        backward_tile<TX, TD, TO, L, CG, GROUP>(mul, n, px, pd, po, wv, st, smem, dw, db);
        group_sync<GROUP>();
        put_back<TO, GROUP>(o, out, row, n, th.lane);
        group_sync<GROUP>();
        now = now + 1 == kTiles ? 0 : now + 1;
    }
    copies_wait<0>();
    if (partial == nullptr) return;
    group_sync<GROUP>();   // every lane's copies have arrived
    float* acc = reinterpret_cast<float*>(mine) + th.lane;
#pragma unroll
    for (int j = 0; j < CG; ++j) acc[j * GROUP] = dw[j], acc[(CG + j) * GROUP] = db[j];
    __syncthreads();
    // every channel's lanes, over the groups and the rows side by side in each, in that order
    float* to = partial + int64_t(blockIdx.x) * 2 * mul;
    for (int i = threadIdx.x; i < 2 * mul; i += blockDim.x) {
        const int which = i / mul, c = i % mul;
        float sum = 0.f;
        for (int k = 0; k < int(blockDim.x) / GROUP; ++k) {
            const float* a = reinterpret_cast<const float*>(memory + k * each) + (which * CG + c / L) * GROUP + c % L;
            for (int u = 0; u < th.G; ++u) sum += a[u * L];
        }
        to[i] = sum;
    }
}

}  // namespace flat
}  // namespace e3gb
