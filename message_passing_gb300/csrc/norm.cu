// Layer norm of rows and irreps norm of node features, forward and backward.
//
// Both normalise segments of K contiguous entries: a row of C channels, or the block b of a
// node's irreps features, 2l+1 rows of mul channels. With the mean mu (0 unless the segment is
// centred), the variance v = sum (x - mu)^2 / K and s = 1 / sqrt(v + eps):
//   xh = (x - mu) s,   y = xh w + b
//   g = w dy,   dx = s (g - [mean g] - xh mean(g xh)),   dw = sum dy xh,   db = sum dy
// where the bracket is there for centred segments only, w is indexed by the channel (and block),
// and the sums of dw and db run over the rows or nodes, and over the 2l+1 rows of a block.
// A norm that mixed degrees l, or the components m of one degree with different scales, or that
// shifted anything but an even scalar, would not commute with rotations and reflections: hence
// one s per (node, block), one w per (block, channel), and mu and b for even scalars only.
//
// The kernels: norm_segments.cuh holds rows of up to about 16,000 entries in registers and
// norm_blocks.cuh the blocks of irreps of up to 256 channels; norm_flat.cuh takes rows whose tensors
// are aligned differently, and the kernels here longer segments. Partial sums of dw and db are added
// by norm_params_sum_kernel in a fixed order.
#include <atomic>
#include <initializer_list>
#include <type_traits>

#include "norm_blocks.cuh"
#include "norm_flat.cuh"
#include "norm_segments.cuh"

namespace e3gb {
namespace {

using segments::group_sum;
using bf16 = __nv_bfloat16;

__device__ __forceinline__ float load_f(const float* p) { return *p; }
__device__ __forceinline__ float load_f(const bf16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store_f(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_f(bf16* p, float v) { *p = __float2bfloat16_rn(v); }

// ------------------------------------------------------------------------------------------
// segments too long for registers: one warp a segment, read again for each pass
// ------------------------------------------------------------------------------------------
template <class TX, class TY>
__global__ void __launch_bounds__(256)
    long_forward_kernel(const __grid_constant__ NormShape sh, const TX* __restrict__ x, const float* __restrict__ w,
                        const float* __restrict__ bias, float eps, TY* __restrict__ y, float2* __restrict__ stats) {
    const int lane = threadIdx.x & 31;
    const int64_t warps = int64_t(gridDim.x) * (blockDim.x >> 5);
    const int64_t n_seg = sh.rows * sh.n_blocks;
    for (int64_t i = int64_t(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5); i < n_seg; i += warps) {
        const int64_t r = i / sh.n_blocks;
        const int b = int(i % sh.n_blocks);
        const int64_t K = int64_t(sh.block_rows[b]) * sh.mul;
        const TX* xs = x + r * sh.x_stride + int64_t(sh.first_row[b]) * sh.mul;
        TY* ys = y + r * sh.y_stride + int64_t(sh.first_row[b]) * sh.mul;
        const bool centred = sh.scalar[b] >= 0;
        float mu = 0.f;
        if (centred) {
            for (int64_t k = lane; k < K; k += 32) mu += load_f(xs + k);
            mu = group_sum<32>(mu, nullptr) / float(K);
        }
        float v = 0.f;
        for (int64_t k = lane; k < K; k += 32) {
            const float d = load_f(xs + k) - mu;
            v = fmaf(d, d, v);
        }
        const float s = rsqrtf(group_sum<32>(v, nullptr) / float(K) + eps);
        if (lane == 0) stats[i] = make_float2(mu, s);
        for (int64_t k = lane; k < K; k += 32) {
            const int64_t q = k % sh.mul;
            float o = (load_f(xs + k) - mu) * s;
            if (w) o *= w[b * sh.mul + q];
            if (bias && centred) o += bias[sh.scalar[b] * sh.mul + q];
            store_f(ys + k, o);
        }
    }
}

template <class TX, class TD, class TO>
__global__ void __launch_bounds__(256)
    long_backward_kernel(const __grid_constant__ NormShape sh, const TX* __restrict__ x, const float* __restrict__ w,
                         const float2* __restrict__ stats, const TD* __restrict__ dy, TO* __restrict__ dx) {
    const int lane = threadIdx.x & 31;
    const int64_t warps = int64_t(gridDim.x) * (blockDim.x >> 5);
    const int64_t n_seg = sh.rows * sh.n_blocks;
    for (int64_t i = int64_t(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5); i < n_seg; i += warps) {
        const int64_t r = i / sh.n_blocks;
        const int b = int(i % sh.n_blocks);
        const int64_t K = int64_t(sh.block_rows[b]) * sh.mul, off = int64_t(sh.first_row[b]) * sh.mul;
        const TX* xs = x + r * sh.x_stride + off;
        const TD* ds = dy + r * sh.dy_stride + off;
        TO* os = dx + r * sh.y_stride + off;
        const float mu = stats[i].x, s = stats[i].y;
        float c1 = 0.f, c2 = 0.f;
        for (int64_t k = lane; k < K; k += 32) {
            const float g = load_f(ds + k) * (w ? w[b * sh.mul + k % sh.mul] : 1.f);
            c1 += g;
            c2 = fmaf(g, (load_f(xs + k) - mu) * s, c2);
        }
        c1 = sh.scalar[b] >= 0 ? group_sum<32>(c1, nullptr) / float(K) : 0.f;
        c2 = group_sum<32>(c2, nullptr) / float(K);
        for (int64_t k = lane; k < K; k += 32) {
            const float g = load_f(ds + k) * (w ? w[b * sh.mul + k % sh.mul] : 1.f);
            const float xh = (load_f(xs + k) - mu) * s;
            store_f(os + k, s * (g - c1 - xh * c2));
        }
    }
}

// partial [gridDim.y][2][n_blocks * mul]: the sums over the rows of part y, one channel a thread
template <class TX, class TD>
__global__ void __launch_bounds__(256)
    long_params_kernel(const __grid_constant__ NormShape sh, const TX* __restrict__ x,
                       const float2* __restrict__ stats, const TD* __restrict__ dy, float* __restrict__ partial) {
    const int64_t n = int64_t(sh.n_blocks) * sh.mul;
    const int64_t c = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
    if (c >= n) return;
    const int b = int(c / sh.mul);
    const int64_t q = c % sh.mul;
    float dw = 0.f, db = 0.f;
    for (int64_t r = blockIdx.y; r < sh.rows; r += gridDim.y) {
        const float2 st = stats[r * sh.n_blocks + b];
        for (int m = 0; m < sh.block_rows[b]; ++m) {
            const int64_t k = int64_t(sh.first_row[b] + m) * sh.mul + q;
            const float d = load_f(dy + r * sh.dy_stride + k);
            dw = fmaf(d, (load_f(x + r * sh.x_stride + k) - st.x) * st.y, dw);
            db += d;
        }
    }
    partial[(2 * int64_t(blockIdx.y)) * n + c] = dw;
    partial[(2 * int64_t(blockIdx.y) + 1) * n + c] = db;
}

// Adds the parts' sums in a fixed order: 8 channels a block (one 32-byte sector of every part), 128 runs of
// parts side by side, since a few hundred parts read one after another would be most of a small call.
__global__ void __launch_bounds__(1024)
    norm_params_sum_kernel(const __grid_constant__ NormShape sh, int parts, const float* __restrict__ partial,
                           float* __restrict__ dw, float* __restrict__ db) {
    __shared__ float smem[2][8][128];
    asm volatile("griddepcontrol.wait;" ::: "memory");   // the kernel before has ended
    const int64_t n = int64_t(sh.n_blocks) * sh.mul;
    const int channel = threadIdx.x & 7, run = threadIdx.x >> 3;
    const int64_t c = int64_t(blockIdx.x) * 8 + channel;
    float a = 0.f, d = 0.f;
    if (c < n) {
#pragma unroll 4
        for (int p = run; p < parts; p += 128) {
            a += partial[2 * int64_t(p) * n + c];
            d += partial[(2 * int64_t(p) + 1) * n + c];
        }
    }
    smem[0][channel][run] = a;
    smem[1][channel][run] = d;
    __syncthreads();
    // a warp for each of the 16 sums
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, which = warp >> 3;
    const int64_t cw = int64_t(blockIdx.x) * 8 + (warp & 7);
    if (warp >= 16 || cw >= n) return;
    const float* from = smem[which][warp & 7];
    const float sum = group_sum<32>((from[lane] + from[lane + 32]) + (from[lane + 64] + from[lane + 96]), nullptr);
    if (lane != 0) return;
    const int b = int(cw / sh.mul);
    if (which == 0 && dw) dw[cw] = sum;
    if (which == 1 && db && sh.scalar[b] >= 0) db[sh.scalar[b] * sh.mul + cw % sh.mul] = sum;
}

// ------------------------------------------------------------------------------------------
// which kernel: by the vectors that types and alignment allow, and by the segment's length
// ------------------------------------------------------------------------------------------
template <int V>
using Int = std::integral_constant<int, V>;
template <bool V>
using Bool = std::integral_constant<bool, V>;

// f(L, NV) for rows of n vectors. Returns false where a row is too long for registers. Many steps from 256
// lanes on: with lanes for the next power of two, a row of 5001 fp32 took 123 us forward and 245 backward
// (64M entries), one of 9001 193 and 289; with these 107, 161 and 95, 146.
template <int VEC, bool ODD, class F>
bool by_length(int64_t n, F&& f) {
    if constexpr (VEC == 8) {
        if (n <= 2) return f(Int<2>{}, Int<1>{}), true;
        if (n <= 4) return f(Int<4>{}, Int<1>{}), true;
        if constexpr (!ODD) {   // odd rows of 5 to 64 vectors of eight go by vectors of four (wide_odd)
            if (n <= 8) return f(Int<4>{}, Int<2>{}), true;
            if (n <= 16) return f(Int<8>{}, Int<2>{}), true;
            if (n <= 32) return f(Int<16>{}, Int<2>{}), true;
            if (n <= 48) return f(Int<16>{}, Int<3>{}), true;
            if (n <= 64) return f(Int<32>{}, Int<2>{}), true;
        }
        if (n <= 128) return f(Int<32>{}, Int<4>{}), true;
        if (n <= 256) return f(Int<256>{}, Int<1>{}), true;
        if (n <= 512) return f(Int<256>{}, Int<2>{}), true;
        if (n <= 768) return f(Int<256>{}, Int<3>{}), true;
        if (n <= 1024) return f(Int<256>{}, Int<4>{}), true;
        if (n <= 1536) return f(Int<512>{}, Int<3>{}), true;
        if (n <= 2048) return f(Int<512>{}, Int<4>{}), true;
    } else {
        if (n <= 2) return f(Int<2>{}, Int<1>{}), true;
        if (n <= 4) return f(Int<4>{}, Int<1>{}), true;
        if (n <= 8) return f(Int<8>{}, Int<1>{}), true;
        if constexpr (ODD) {
            if (n <= 12) return f(Int<4>{}, Int<3>{}), true;
        }
        if (n <= 16) return f(Int<8>{}, Int<2>{}), true;
        if (n <= 24) return f(Int<8>{}, Int<3>{}), true;
        if (n <= 32) return f(Int<8>{}, Int<4>{}), true;
        if (n <= 48) return f(Int<16>{}, Int<3>{}), true;
        if (n <= 64) return f(Int<16>{}, Int<4>{}), true;
        if (n <= 96) return f(Int<32>{}, Int<3>{}), true;
        if (n <= 128) return f(Int<32>{}, Int<4>{}), true;
        if (n <= 256) return f(Int<32>{}, Int<8>{}), true;
        if (n <= 512) return f(Int<256>{}, Int<2>{}), true;
        if (n <= 1024) return f(Int<256>{}, Int<4>{}), true;
        if (n <= 1280) return f(Int<256>{}, Int<5>{}), true;
        if (n <= 1536) return f(Int<512>{}, Int<3>{}), true;
        if (n <= 2048) return f(Int<512>{}, Int<4>{}), true;
        if (n <= 2560) return f(Int<512>{}, Int<5>{}), true;
        if (n <= 3072) return f(Int<512>{}, Int<6>{}), true;
        if (n <= 4096) return f(Int<512>{}, Int<8>{}), true;
    }
    return false;
}

// f(L, MV, CG) for blocks of n vectors of channels
template <int VEC, class F>
bool by_channels(int64_t n, F&& f) {
    if constexpr (VEC > 1) {
        if (n == 1) return f(Int<2>{}, Int<2>{}, Int<1>{}), true;
        if (n == 2) return f(Int<8>{}, Int<2>{}, Int<1>{}), true;
        if (n <= 4) return f(Int<4>{}, Int<4>{}, Int<1>{}), true;
    }
    if (n <= 8) return f(Int<8>{}, Int<8>{}, Int<1>{}), true;
    if (n <= 16) return f(Int<16>{}, Int<16>{}, Int<1>{}), true;
    if (n <= 32) return f(Int<32>{}, Int<32>{}, Int<1>{}), true;
    if (n <= 64) return f(Int<32>{}, Int<32>{}, Int<2>{}), true;
    if constexpr (VEC == 1) {
        if (n <= 128) return f(Int<32>{}, Int<32>{}, Int<4>{}), true;
        if (n <= 256) return f(Int<32>{}, Int<32>{}, Int<8>{}), true;
    }
    return false;
}

// f(L, CG, group) for the flat kernels
template <class F>
bool by_flat_row(int64_t C, F&& f) {
    if (C <= 8) return f(Int<8>{}, Int<1>{}, Int<32>{}), true;
    if (C <= 32) return f(Int<8>{}, Int<4>{}, Int<32>{}), true;
    if (C <= 128) return f(Int<32>{}, Int<4>{}, Int<32>{}), true;
    if (C <= 512) return f(Int<32>{}, Int<16>{}, Int<32>{}), true;
    if (C <= 2048) return f(Int<256>{}, Int<8>{}, Int<256>{}), true;
    if (C <= 8192) return f(Int<512>{}, Int<16>{}, Int<512>{}), true;
    return false;
}

// a tensor of rows of n entries for the flat kernels, L lanes to a row
template <class T>
flat::Rows flat_rows(const T* p, int64_t rows, int64_t n, int64_t stride, int L) {
    flat::Rows r{};
    r.base = reinterpret_cast<char*>(const_cast<T*>(p));
    r.stride = stride * int64_t(sizeof(T));
    r.row = int(n * int64_t(sizeof(T)));
    r.end = r.base + (rows - 1) * r.stride + r.row;
    r.units = reinterpret_cast<uintptr_t>(p) % 16 == 0 && r.stride % 16 == 0 && r.row % 16 == 0;
    r.pitch = r.row;
    if (r.units && L < 32)   // rows side by side start L entries apart, modulo the 128 bytes of the banks
        while (r.pitch % 128 != (L * int(sizeof(T))) % 128) r.pitch += 16;
    return r;
}
// rows of a tile: about 4 KB of inputs, whole steps of G rows; one where the rows of a tensor that is not
// made of 16-byte units do not follow one another
int flat_tile(std::initializer_list<flat::Rows*> ts, int inputs, int G, int group) {
    bool follow = true;
    for (const flat::Rows* r : ts) follow = follow && (r->units || r->stride == r->row);
    const int n = 4096 / inputs / G * G;
    const int tile = group > 32 || !follow ? 1 : n < G ? G : n > 64 ? 64 : n;
    for (flat::Rows* r : ts) r->slot = (r->units ? tile * r->pitch : tile * r->row + 16) / 16 * 16 + 16;
    return tile;
}

constexpr int kMaxSmem = 226 * 1024;   // of a block, less its static part
// threads of a block whose warps take `each` bytes: two blocks to a multiprocessor where they fit
int flat_threads(int each) {
    for (int t = 256; t > 32; t /= 2)
        if (each * (t / 32) <= kMaxSmem / 2) return t;
    return 32;
}

// Rows of a lane's ring in shared memory: two or three. Three keep loads going while a row's sum goes through its
// shuffles or its barrier, two leave the L1 cache and the registers more. Measured, 64M entries, with two and
// with three:
//   forward, three: bf16 by vectors of eight with three or more a lane (768: 55, 49 us; 1024: 48, 44; 264: 48, 43, but
//     384: 42, 45) and bf16 of rows shared by warps (2048: 51, 47; 4096: 52, 46; 6000: 48, 44; to fp32 66, 61); odd
//     rows of up to 256 lanes (fp32 77: 90, 83; 321: 90, 84; 1999: 87, 83);
//   forward, two: other fp32 (64: 83, 86; 768: 78, 88; 2048: 77, 92; 5000: 78, 94; but 6000: 92, 83), and a warp with
//     eight vectors of four (odd fp32 999: 88, 132; bf16 to fp32 1024: 61, 66, but 700: 68, 63);
//   backward, three: rows of 256 lanes (fp32 4096: 127, 121; 5000: 131, 122; bf16 2048: 90, 84; 4096: 93, 79) but for
//     fp32 by two vectors (2048, 134M entries: 246, 259); fp32 by four vectors in 512 lanes (8192: 135, 130; but
//     7000: 123, 135);
//   backward, two: other rows (fp32 64: 126, 125; 512: 122, 125; 6000: 125, 141; bf16 1024, 134M entries: 126, 136;
//     16384: 114, 134; but 384: 69, 63) and odd ones (fp32 77: 119, 143; 3001: 179, 225; bf16 321: 119, 147; 5001: 147,
//     168; 13001: 187, 227).
template <class TX, int VEC, int L, int NV, bool ODD>
constexpr int forward_rows = (ODD ? L <= 256 && NV <= 4 : sizeof(TX) == 2 && (L > 32 || (VEC == 8 && NV >= 3))) ? 3 : 2;
template <class TX, class TD, int VEC, int L, int NV, bool ODD>
constexpr int backward_rows =
    !ODD && (sizeof(TX) + sizeof(TD) < 8 ? L == 256 : (L == 256 && NV > 2) || (L == 512 && NV == 4)) ? 3 : 2;
// as many of those as a block has room for
constexpr int row_stages(int slot, int want) { return want * slot <= 216 * 1024 ? want : 2 * slot <= 216 * 1024 ? 2 : 1; }

int resident(const void* kernel, int threads, int smem) { return grid_for(kernel, threads, 1, int64_t(1) << 40, smem); }

// thread blocks for `rows` rows, `per` a block; `unit`: what their number is a multiple of, unless every
// block has one round only
int blocks_for(int64_t rows, int per, int unit, int most) {
    const int64_t need = (rows + per - 1) / per;
    return int(need < most ? need : most / unit * unit);
}

// whether vectors of VEC entries of the tensors lie over one another, and whether rows are whole vectors
template <class A, class B>
bool same_shift(const A* a, int64_t as, const B* b, int64_t bs, int vec) {
    return (reinterpret_cast<uintptr_t>(a) / sizeof(A)) % vec == (reinterpret_cast<uintptr_t>(b) / sizeof(B)) % vec &&
           as % vec == bs % vec;
}
template <class T>
bool vectors_fit(const T* p, int64_t stride, int vec) {
    return reinterpret_cast<uintptr_t>(p) % (vec * sizeof(T)) == 0 && stride % vec == 0;
}

// lifts a kernel's limit of shared memory, once a device (TAG: one for each kernel)
template <class TAG>
cudaError_t allow_smem(TAG, const void* kernel) {
    static std::atomic<uint64_t> set{0};
    int dev = 0;
    cudaGetDevice(&dev);
    const uint64_t bit = uint64_t(1) << (dev & 63);
    if (set.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
    if (e == cudaSuccess) set.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

constexpr int64_t kL2Bytes = 126 * 1000 * 1000;

// Irreps of 4 and 8 channels in fp32 (rows of 16 and 32 bytes) whose bytes stay in the L2 cache anyway are loaded as
// read once, larger ones are kept in the caches. Measured, read once and kept:
//   forward, 8 channels, up to what x and y hold together (120,000 x 16: 23, 26 us; 200,000 x 9: 25, 28; 50,000 x 31:
//     17, 20; above, 150,000 x 16: 33, 31; 200,000 x 16: 44, 38; 250,000 x 9: 36, 34);
//   forward, 4 channels, up to three quarters by x (400,000 x 9: 29, 32; 600,000 x 9: 45, 53; above, 800,000 x 9: 90, 73);
//   backward, 8 channels, up to x and dy (75,000 x 16: 26, 29; 100,000 x 16: 31, 34; 200,000 x 9: 46, 49; above, 150,000
//     x 16: 53, 46; 250,000 x 9: 58, 52).
template <class TX, int VEC, int MV>
constexpr bool read_once = VEC == 4 && MV <= 2 && sizeof(TX) == 4;
template <class TX, class TY, int L, int MV>
bool forward_once(int64_t entries) {
    return MV < L ? entries * int64_t(sizeof(TX) + sizeof(TY)) <= kL2Bytes
                  : entries * int64_t(sizeof(TX)) <= kL2Bytes / 4 * 3;
}

// Nodes, a multiple of unit between half of `about` and twice it, that share rows out most evenly among
// thread blocks that take so many at a time.
int64_t block_tile(int64_t rows, int64_t blocks, int unit, int about) {
    int64_t best = about, least = INT64_MAX;
    for (int64_t t = about / 2; t <= 2 * about; t += unit) {
        const int64_t most = (rows + blocks * t - 1) / (blocks * t) * t;
        if (most < least || (most == least && t <= about)) best = t, least = most;
    }
    return best;
}

bool is_rows(const NormShape& sh) { return sh.n_blocks == 1 && sh.block_rows[0] == 1 && sh.scalar[0] == 0; }

template <class T>
segments::Tensor<T> rows_of(T* p, int64_t stride, const NormShape& sh) {
    return {p, stride, p + (sh.rows - 1) * stride + sh.mul};
}

// Whether odd bf16 rows of n entries go by vectors of eight: between these bounds vectors of four waste
// fewer lanes on the two ends (backward, 64M entries, by eight and by four: 143, 117 us at 77; 120, 152 at 999).
bool wide_odd(int64_t n) { return n < 24 || n > 512; }

// vectors that a row of n entries can touch
int64_t vectors_of(int64_t n, int vec, bool odd) { return odd ? (n + 2 * vec - 2) / vec : n / vec; }

template <class TX, class TY>
cudaError_t forward(const NormShape& sh, const TX* xc, const float* w, const float* bias, float eps, TY* y,
                    float2* stats, cudaStream_t s) {
    TX* x = const_cast<TX*>(xc);
    cudaError_t e = cudaSuccess;
    const auto tensor = [&](auto* p, int64_t stride) { return rows_of(p, stride, sh); };
    const auto rows = [&](auto vec, auto odd) {
        constexpr int VEC = decltype(vec)::value;
        constexpr bool ODD = decltype(odd)::value;
        return by_length<VEC, ODD>(vectors_of(sh.mul, VEC, ODD), [&](auto l, auto nv) {
            constexpr int L = decltype(l)::value, NV = decltype(nv)::value, T = segments::kThreads<L>;
            constexpr int slot = segments::Ring<TX, VEC, L, NV, ODD>::kBytes, S = row_stages(slot, forward_rows<TX, VEC, L, NV, ODD>), smem = slot * S;
            auto* k = segments::forward_kernel<TX, TY, VEC, L, NV, S, ODD>;
            e = allow_smem([] {}, (const void*)k);
            if (e != cudaSuccess) return;
            const int grid = blocks_for(sh.rows, T / L, L == T ? VEC : 1, resident((const void*)k, T, smem));
            k<<<grid, T, smem, s>>>(sh.rows, int(sh.mul), tensor(x, sh.x_stride), tensor(y, sh.y_stride), w, bias, eps, stats);
        });
    };
    const auto flat_rows_kernel = [&] {
        return by_flat_row(sh.mul, [&](auto l, auto cg, auto group) {
            constexpr int L = decltype(l)::value, GROUP = decltype(group)::value;
            flat::Rows rx = flat_rows(x, sh.rows, sh.mul, sh.x_stride, L), ry = flat_rows(y, sh.rows, sh.mul, sh.y_stride, L);
            const int tile = flat_tile({&rx, &ry}, rx.row, GROUP / L, GROUP), each = flat::kTiles * rx.slot + ry.slot;
            const int threads = GROUP > 32 ? GROUP : flat_threads(each), smem = each * (threads / GROUP);
            auto* k = flat::forward_kernel<TX, TY, L, decltype(cg)::value, GROUP>;
            e = allow_smem([] {}, (const void*)k);
            if (e != cudaSuccess) return;
            const int grid = grid_for((const void*)k, threads, int64_t(threads / GROUP) * tile, sh.rows, smem);
            k<<<grid, threads, smem, s>>>(sh, rx, ry, tile, w, bias, eps, stats);
        });
    };
    const auto blocks = [&](auto vec) {
        constexpr int VEC = decltype(vec)::value;
        return by_channels<VEC>(sh.mul / VEC, [&](auto l, auto mv, auto cg) {
            constexpr int L = decltype(l)::value, MV = decltype(mv)::value, CG = decltype(cg)::value;
            const auto launch = [&](auto* k, int nodes) {
                k<<<grid_for((const void*)k, 256, nodes * 256 / L, sh.rows, 0), 256, 0, s>>>(sh, x, w, bias, eps, y, stats);
            };
            constexpr bool once = read_once<TX, VEC, MV>;
            if constexpr (blocks::kPairs<TX, TY, VEC, L, MV, CG>)
                launch(blocks::irreps_forward_pairs_kernel<TX, TY, VEC, L, MV, CG>, 2);
            else if (once && forward_once<TX, TY, L, MV>(sh.rows * sh.x_stride))
                launch(blocks::irreps_forward_kernel<TX, TY, VEC, L, MV, CG, !once>, 1);
            else
                launch(blocks::irreps_forward_kernel<TX, TY, VEC, L, MV, CG, true>, 1);
        });
    };
    const auto fits = [&](int vec) {
        return sh.mul % vec == 0 && vectors_fit(x, sh.x_stride, vec) && vectors_fit(y, sh.y_stride, vec);
    };
    const auto over = [&](int vec) { return same_shift(x, sh.x_stride, y, sh.y_stride, vec); };
    constexpr bool narrow = sizeof(TX) == 2 && sizeof(TY) == 2;
    bool done = false;
    if (is_rows(sh)) {
        if constexpr (narrow) {
            if (fits(8)) done = rows(Int<8>{}, Bool<false>{});
        }
        if (!done && fits(4)) done = rows(Int<4>{}, Bool<false>{});
        if constexpr (narrow) {
            if (!done && wide_odd(sh.mul) && over(8)) done = rows(Int<8>{}, Bool<true>{});
        }
        if (!done && over(4)) done = rows(Int<4>{}, Bool<true>{});
        if (!done) done = flat_rows_kernel();
    } else {
        done = fits(4) ? blocks(Int<4>{}) : blocks(Int<1>{});
    }
    if (!done) {
        auto* k = long_forward_kernel<TX, TY>;
        k<<<grid_for((const void*)k, 256, 8, sh.rows * sh.n_blocks, 0), 256, 0, s>>>(sh, x, w, bias, eps, y, stats);
    }
    return e != cudaSuccess ? e : cudaGetLastError();
}

// parts of the parameters' sums that a workspace has room for
int most_parts(const NormShape& sh) {
    const int64_t n = int64_t(sh.n_blocks) * sh.mul;
    const int64_t room = n <= 1024 ? 8 * 152 : n <= 16384 ? (8 * 152 * 1024 / n > 152 ? 8 * 152 * 1024 / n : 152) : (8 * 152 * 256 + n - 1) / n + 8;
    const int64_t rows = (sh.rows + 7) / 8 * 8;
    const int64_t most = (rows < room ? rows : room) / 8 * 8;
    return int(most < 8 ? 8 : most);
}

template <class TX, class TD, class TO>
cudaError_t backward(const NormShape& sh, const TX* xc, const float* w, const float2* stats, const TD* dyc, TO* dx,
                     float* dw, float* db, float* ws, cudaStream_t s) {
    TX* x = const_cast<TX*>(xc);
    TD* dy = const_cast<TD*>(dyc);
    const bool params = dw != nullptr || db != nullptr;
    const int64_t n = int64_t(sh.n_blocks) * sh.mul;
    float* partial = params ? ws : nullptr;
    int parts = 0;
    cudaError_t e = cudaSuccess;
    const auto tensor = [&](auto* p, int64_t stride) { return rows_of(p, stride, sh); };
    if (sh.rows > 0) {
        const int most = most_parts(sh);
        const auto rows = [&](auto vec, auto odd) {
            constexpr int VEC = decltype(vec)::value;
            constexpr bool ODD = decltype(odd)::value;
            return by_length<VEC, ODD>(vectors_of(sh.mul, VEC, ODD), [&](auto l, auto nv) {
                constexpr int L = decltype(l)::value, NV = decltype(nv)::value, T = segments::kThreads<L>;
                constexpr int slot = segments::Ring<TX, VEC, L, NV, ODD>::kBytes + segments::Ring<TD, VEC, L, NV, ODD>::kBytes + 8 * T;
                constexpr int S = row_stages(slot, backward_rows<TX, TD, VEC, L, NV, ODD>), smem = slot * S;
                auto* k = segments::backward_kernel<TX, TD, TO, VEC, L, NV, S, ODD>;
                e = allow_smem([] {}, (const void*)k);
                if (e != cudaSuccess) return;
                const int cap = resident((const void*)k, T, smem);
                parts = blocks_for(sh.rows, T / L, L == T ? VEC : 1, cap < most ? cap : most);
                k<<<parts, T, smem, s>>>(sh.rows, int(sh.mul), tensor(x, sh.x_stride), tensor(dy, sh.dy_stride),
                                         tensor(dx, sh.y_stride), w, stats, partial);
            });
        };
        const auto flat_rows_kernel = [&] {
            return by_flat_row(sh.mul, [&](auto l, auto cg, auto group) {
                constexpr int L = decltype(l)::value, CG = decltype(cg)::value, GROUP = decltype(group)::value;
                flat::Rows rx = flat_rows(x, sh.rows, sh.mul, sh.x_stride, L), rd = flat_rows(dy, sh.rows, sh.mul, sh.dy_stride, L),
                           ro = flat_rows(dx, sh.rows, sh.mul, sh.y_stride, L);
                const int tile = flat_tile({&rx, &rd, &ro}, rx.row + rd.row, GROUP / L, GROUP);
                const int tiles = flat::kTiles * (rx.slot + rd.slot + (tile * 8 + 15) / 16 * 16) + ro.slot;
                const int sums = 2 * CG * GROUP * 4, each = tiles > sums ? tiles : sums;
                const int threads = GROUP > 32 ? GROUP : flat_threads(each), smem = each * (threads / GROUP);
                auto* k = flat::backward_kernel<TX, TD, TO, L, CG, GROUP>;
                e = allow_smem([] {}, (const void*)k);
                if (e != cudaSuccess) return;
                const int grid = grid_for((const void*)k, threads, int64_t(threads / GROUP) * tile, sh.rows, smem);
                parts = grid < most ? grid : most;
                k<<<parts, threads, smem, s>>>(sh, rx, rd, ro, tile, each, w, stats, partial);
            });
        };
        const auto blocks = [&](auto vec) {
            constexpr int VEC = decltype(vec)::value;
            return by_channels<VEC>(sh.mul / VEC, [&](auto l, auto mv, auto cg) {
                constexpr int L = decltype(l)::value;
                constexpr int MV = decltype(mv)::value, CG = decltype(cg)::value, unit = 256 / L;
                int sums = 0;
                for (int b = 0; b < sh.n_blocks; ++b) sums += sh.scalar[b] >= 0 ? 2 : 1;
                const int smem = params ? sums * CG * VEC * 256 * int(sizeof(float)) : 0;
                const auto launch = [&](auto* k, auto tag) {
                    e = allow_smem(tag, (const void*)k);
                    if (e != cudaSuccess) return;
                    const int grid = grid_for((const void*)k, 256, 2 * unit, sh.rows, smem);
                    parts = grid < most ? grid : most;
                    const bool one = (VEC == 4 && L == 32 && sizeof(TX) == 4 && sh.mul % 32 == 0) || CG == 8;
                    const int64_t tile = one ? (sh.rows + parts - 1) / parts
                                             : block_tile(sh.rows, parts, unit, VEC == 4 && MV == L ? 2 * unit : 4 * unit);
                    k<<<parts, 256, smem, s>>>(sh, x, w, stats, dy, dx, partial, tile);
                };
                constexpr bool once = MV < L && read_once<TX, VEC, MV>;
                if (once && sh.rows * sh.x_stride * int64_t(sizeof(TX) + sizeof(TD)) <= kL2Bytes)
                    launch(blocks::irreps_backward_kernel<TX, TD, TO, VEC, L, MV, CG, !once>, [] {});
                else
                    launch(blocks::irreps_backward_kernel<TX, TD, TO, VEC, L, MV, CG, true>, [] {});
            });
        };
        const auto fits = [&](int vec) {
            return sh.mul % vec == 0 && vectors_fit(x, sh.x_stride, vec) && vectors_fit(dy, sh.dy_stride, vec) &&
                   vectors_fit(dx, sh.y_stride, vec);
        };
        const auto over = [&](int vec) {
            return same_shift(x, sh.x_stride, dy, sh.dy_stride, vec) && same_shift(x, sh.x_stride, dx, sh.y_stride, vec);
        };
        constexpr bool narrow = sizeof(TX) == 2 && sizeof(TD) == 2 && sizeof(TO) == 2;
        bool done = false;
        if (is_rows(sh)) {
            if constexpr (narrow) {
                if (fits(8)) done = rows(Int<8>{}, Bool<false>{});
            }
            if (!done && fits(4)) done = rows(Int<4>{}, Bool<false>{});
            if constexpr (narrow) {
                if (!done && wide_odd(sh.mul) && over(8)) done = rows(Int<8>{}, Bool<true>{});
            }
            if (!done && over(4)) done = rows(Int<4>{}, Bool<true>{});
            if (!done) done = flat_rows_kernel();
        } else {
            done = fits(4) ? blocks(Int<4>{}) : blocks(Int<1>{});
        }
        if (!done) {
            auto* k = long_backward_kernel<TX, TD, TO>;
            k<<<grid_for((const void*)k, 256, 8, sh.rows * sh.n_blocks, 0), 256, 0, s>>>(sh, x, w, stats, dy, dx);
            if (params) {
                parts = most;
                long_params_kernel<TX, TD><<<dim3(unsigned((n + 255) / 256), most), 256, 0, s>>>(sh, x, stats, dy, ws);
            }
        }
        if (e == cudaSuccess) e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    if (!params) return cudaSuccess;
    // its launch overlaps the end of the kernel before it, whose blocks allow that (launch_dependents)
    cudaLaunchConfig_t config{};
    config.gridDim = dim3(unsigned((n + 7) / 8));
    config.blockDim = dim3(1024);
    config.stream = s;
    cudaLaunchAttribute early{};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    config.attrs = &early;
    config.numAttrs = sh.rows > 0 ? 1 : 0;
    return cudaLaunchKernelEx(&config, norm_params_sum_kernel, sh, parts, (const float*)ws, dw, db);
}

}  // namespace

#if E3GB_PART == 0
size_t norm_backward_workspace_bytes(const NormShape& sh) {
    return size_t(most_parts(sh)) * 2 * size_t(sh.n_blocks) * size_t(sh.mul) * sizeof(float);
}

cudaError_t norm_forward(const NormShape& sh, const void* x, int x_bf16, const float* w, const float* bias,
                         float eps, void* y, int y_bf16, float* stats, cudaStream_t s) {
    const auto go = [&](auto tx, auto ty) {
        using TX = decltype(tx);
        using TY = decltype(ty);
        return forward<TX, TY>(sh, (const TX*)x, w, bias, eps, (TY*)y, (float2*)stats, s);
    };
    if (x_bf16) return y_bf16 ? go(bf16{}, bf16{}) : go(bf16{}, 0.f);
    return y_bf16 ? go(0.f, bf16{}) : go(0.f, 0.f);
}

cudaError_t norm_backward(const NormShape& sh, const void* x, int x_bf16, const float* w, const float* stats,
                          const void* dy, int dy_bf16, void* dx, int dx_bf16, float* dw, float* db, float* ws,
                          cudaStream_t s) {
    static NormBackward* const by_types[8] = {norm_backward_fff, norm_backward_ffb, norm_backward_fbf, norm_backward_fbb,
                                              norm_backward_bff, norm_backward_bfb, norm_backward_bbf, norm_backward_bbb};
    return by_types[(x_bf16 ? 4 : 0) + (dy_bf16 ? 2 : 0) + (dx_bf16 ? 1 : 0)](sh, x, w, stats, dy, dx, dw, db, ws, s);
}
#else
// the backward for one set of types of x, dy and dx (its own translation unit each)
#define E3GB_BACKWARD(NAME, X, D, O)                                                                                   \
    cudaError_t NAME(const NormShape& sh, const void* x, const float* w, const float* stats, const void* dy, void* dx, \
                     float* dw, float* db, float* ws, cudaStream_t s) {                                                \
        return backward<X, D, O>(sh, (const X*)x, w, (const float2*)stats, (const D*)dy, (O*)dx, dw, db, ws, s);       \
    }
#if E3GB_PART == 1
E3GB_BACKWARD(norm_backward_fff, float, float, float)
#elif E3GB_PART == 2
E3GB_BACKWARD(norm_backward_ffb, float, float, bf16)
#elif E3GB_PART == 3
E3GB_BACKWARD(norm_backward_fbf, float, bf16, float)
#elif E3GB_PART == 4
E3GB_BACKWARD(norm_backward_fbb, float, bf16, bf16)
#elif E3GB_PART == 5
E3GB_BACKWARD(norm_backward_bff, bf16, float, float)
#elif E3GB_PART == 6
E3GB_BACKWARD(norm_backward_bfb, bf16, float, bf16)
#elif E3GB_PART == 7
E3GB_BACKWARD(norm_backward_bbf, bf16, bf16, float)
#else
E3GB_BACKWARD(norm_backward_bbb, bf16, bf16, bf16)
#endif
#undef E3GB_BACKWARD
#endif

}  // namespace e3gb
