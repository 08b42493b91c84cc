// An AdamW step over many tensors in one launch, with 32-bit or 8-bit moments.
//
//   m = b1 m + (1 - b1) g,   v = b2 v + (1 - b2) g^2,
//   p = p (1 - lr wd) - lr / (1 - b1^t) m / (sqrt(v) / sqrt(1 - b2^t) + eps),
// with g scaled by min(1, max_norm / |g|) first where the step clips; |g| is the 2-norm of all
// gradients together. A step whose norm is not finite changes nothing.
//
// 8-bit moments: blocks of 256 entries share a power of two, chosen so that the block's largest
// finite entry takes the top binade of the format. m has sign, 4 exponent and 3 mantissa bits; v,
// whose range is the square of m's, 5 exponent and 2 mantissa bits. Both are rounded up with the
// probability of the part cut off: with b2 = 0.999 a step moves v by about a thousandth, and
// rounding to nearest, with codes 14-25% apart, would never move it. The random bits are a fixed
// function of (seed, step, entry), so that a step can be repeated. A positive v never rounds to
// zero: its root under m's smallest code would make a step of m / eps. The update itself takes
// the moments before they are rounded.
//
// The moments' arithmetic is written as single rounded operations, not fused: a code is then the
// same wherever the same formula is evaluated in IEEE fp32, one entry at a time.
//
// Bound by memory: an entry costs 28 bytes with 32-bit moments and fp32 gradients, 14 with 8-bit
// moments and bf16 gradients. A thread block takes a run of neighbouring chunks of 4096 entries.
// Measured: 134M entries, fp32 gradients, bf16 copies and clipping 711 us (the step itself 96% of the
// copy rate, the norm's second read of the gradients 100 us); 200M entries with 8-bit moments and
// bf16 gradients 458 us (91%; the arithmetic units are 60-70% busy, so the loads have to come early).
#include "adamw.cuh"
#include "async_copy.cuh"

#include <cuda_fp8.h>

#include <atomic>

namespace e3gb {
int grid_for(const void* kernel, int block, int64_t per_block, int64_t units, int smem);
namespace {

constexpr int kThreads = 256;

struct Gradients {
    const void* g[kAdamwLaunch];
};

__device__ __forceinline__ float load_f(const float* p) { return *p; }
__device__ __forceinline__ float load_f(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void unpack(const float4& r, float (&f)[4]) { f[0] = r.x, f[1] = r.y, f[2] = r.z, f[3] = r.w; }
__device__ __forceinline__ void unpack(const uint2& r, float (&f)[4]) {
    f[0] = __uint_as_float(r.x << 16), f[1] = __uint_as_float(r.x & 0xffff0000u);
    f[2] = __uint_as_float(r.y << 16), f[3] = __uint_as_float(r.y & 0xffff0000u);
}
template <class TG>
struct Raw4;
template <>
struct Raw4<float> { using type = float4; };
template <>
struct Raw4<__nv_bfloat16> { using type = uint2; };
__device__ __forceinline__ uint32_t pair(float a, float b) {
    const __nv_bfloat162 t = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&t);
}

// A sum kept as the unevaluated sum of two fp32 numbers: about 48 bits without the few fp64 units.
__device__ __forceinline__ float2 add(float2 a, float2 b) {
    const float s = __fadd_rn(a.x, b.x), t = __fsub_rn(s, a.x);
    const float err = __fadd_rn(__fsub_rn(a.x, __fsub_rn(s, t)), __fsub_rn(b.x, t));
    return make_float2(s, __fadd_rn(err, __fadd_rn(a.y, b.y)));
}
// over the block, for every thread
__device__ __forceinline__ float2 block_sum(float2 v, float2* smem) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v = add(v, make_float2(__shfl_xor_sync(0xffffffffu, v.x, o), __shfl_xor_sync(0xffffffffu, v.y, o)));
    if ((threadIdx.x & 31) == 0) smem[threadIdx.x >> 5] = v;
    __syncthreads();
    v = smem[0];
    for (int i = 1; i < kThreads / 32; ++i) v = add(v, smem[i]);
    return v;
}

template <class TG>
__device__ __forceinline__ bool aligned4(const TG* g) { return reinterpret_cast<uintptr_t>(g) % (4 * sizeof(TG)) == 0; }

// The chunks of a launch, cut into `runs` of neighbouring ones, and a run into stretches of one
// tensor: f(tensor, number of the tensor, first entry, one past the last). Inside a stretch every
// address is an offset, so that loads can be issued far ahead.
template <class F>
__device__ __forceinline__ void stretches(const AdamwTensor* __restrict__ tensors, const int32_t* __restrict__ chunk_tensor,
                                          int chunk0, int chunks, int run, int runs, F&& f) {
    int c = chunk0 + int(int64_t(chunks) * run / runs);
    const int end = chunk0 + int(int64_t(chunks) * (run + 1) / runs);
    if (c >= end) return;
    for (int t = chunk_tensor[c]; c < end; ++t) {
        const AdamwTensor a = tensors[t];
        const int64_t first = int64_t(c - a.first_chunk) * kAdamwChunk, rest = int64_t(end - a.first_chunk) * kAdamwChunk;
        const int64_t last = rest < a.numel ? rest : a.numel;
        if (first >= last) continue;   // a tensor without entries
        f(a, t, first, last);
        c += int((last - first + kAdamwChunk - 1) / kAdamwChunk);
    }
}

// partial[blockIdx.x] = the sum of g^2 over every kNormSplit-th chunk of a run, kNormSplit blocks to a
// run of the step. A stretch goes from its end to its start: the step begins where the norm ended,
// with those gradients still in L2.
constexpr int kNormSplit = 4;
template <class TG>
__global__ void __launch_bounds__(kThreads)
    adamw_norm_kernel(const AdamwTensor* __restrict__ tensors, const int32_t* __restrict__ chunk_tensor, int tensor0,
                      int chunk0, int chunks, const __grid_constant__ Gradients grads, float2* __restrict__ partial) {
    __shared__ float2 smem[kThreads / 32];
    using R = typename Raw4<TG>::type;
    const int run = blockIdx.x / kNormSplit, split = blockIdx.x % kNormSplit;
    float2 total = make_float2(0.f, 0.f);
    stretches(tensors, chunk_tensor, chunk0, chunks, run, gridDim.x / kNormSplit,
              [&](const AdamwTensor&, int t, int64_t first, int64_t last) {
        const TG* g = static_cast<const TG*>(grads.g[t - tensor0]);
        if (g == nullptr) return;
        const int64_t end = (last - 1 - first) / kAdamwChunk;
        if (!aligned4(g)) {
            for (int64_t c = end - (end + kNormSplit - split) % kNormSplit; c >= 0; c -= kNormSplit) {
                const int64_t at = first + c * kAdamwChunk, rest = last - at;
                float sum = 0.f;
                for (int i = threadIdx.x; i < (rest < kAdamwChunk ? int(rest) : kAdamwChunk); i += kThreads)
                    sum = fmaf(load_f(g + at + i), load_f(g + at + i), sum);
                total = add(total, make_float2(sum, 0.f));
            }
            return;
        }
        constexpr int V = kAdamwChunk / kThreads / 4;
        const int64_t whole = last & ~int64_t(3);
        if (split == 0 && last - whole > int(threadIdx.x)) {
            const float f = load_f(g + whole + threadIdx.x);
            total = add(total, make_float2(f * f, 0.f));
        }
        for (int64_t c = end - (end + kNormSplit - split) % kNormSplit; c >= 0; c -= kNormSplit) {
            R r[V];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int64_t i = first + c * kAdamwChunk + (j * kThreads + int(threadIdx.x)) * 4;
                r[j] = R{};
                if (i < whole) r[j] = *reinterpret_cast<const R*>(g + i);
            }
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                float f[4];
                unpack(r[j], f);
#pragma unroll
                for (int k = 0; k < 4; ++k) sum = fmaf(f[k], f[k], sum);
            }
            total = add(total, make_float2(sum, 0.f));
        }
    });
    total = block_sum(total, smem);
    if (threadIdx.x == 0) partial[blockIdx.x] = total;
}

__device__ __forceinline__ void moments(float g, float& m, float& v, float beta1, float beta2, const AdamwRates& r) {
    m = __fadd_rn(__fmul_rn(m, beta1), __fmul_rn(g, r.rest1));
    v = __fadd_rn(__fmul_rn(v, beta2), __fmul_rn(__fmul_rn(g, g), r.rest2));
}
__device__ __forceinline__ float max_or_nan(float a, float b) {
    float m;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
    return m;
}
// Root and reciprocal are the units' approximations, each within two units of 2^-24 relative. The root takes
// subnormal numbers as they are: a v of 1e-40 (gradients of 1e-19) taken for zero would leave eps alone
// under m. The reciprocal's operand is a normal number, at least eps >= 1e-30.
__device__ __forceinline__ float update(float p, float m, float v, float2 keep, const AdamwRates& r) {
    float root, quotient;
    asm("sqrt.approx.f32 %0, %1;" : "=f"(root) : "f"(v));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(quotient) : "f"(fmaf(root, r.root, r.eps)));
    return fmaf(p, keep.x, fmaf(p, keep.y, -(m * quotient * r.step_size)));
}

// 1 - lr wd as the sum of two fp32 numbers: one of them would round an lr wd of 1e-7 to 1.2e-7 and one of 2e-8
// to nothing, at every step the same way.
__device__ __forceinline__ float2 keeps(float lr, float decay) {
    const float d = __fmul_rn(lr, decay), rest = fmaf(lr, decay, -d);
    const float hi = __fsub_rn(1.f, d), t = __fsub_rn(hi, 1.f);
    return make_float2(hi, __fsub_rn(__fsub_rn(__fsub_rn(1.f, __fsub_rn(hi, t)), __fadd_rn(d, t)), rest));
}

// four entries of m and v (8-bit codes) in units of their block's scales; both formats are subsets
// of fp16, the second its upper byte
__device__ __forceinline__ void from_codes(uint32_t mc, uint32_t vc, float (&m)[4], float (&v)[4]) {
    const __half2_raw m0 = __nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(mc & 0xffffu), __NV_E4M3);
    const __half2_raw m1 = __nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(mc >> 16), __NV_E4M3);
    const float2 a = __half22float2(__half2(m0)), b = __half22float2(__half2(m1));
    m[0] = a.x, m[1] = a.y, m[2] = b.x, m[3] = b.y;
    const uint32_t v0 = __byte_perm(vc, 0u, 0x1404), v1 = __byte_perm(vc, 0u, 0x3424);
    const float2 c = __half22float2(*reinterpret_cast<const __half2*>(&v0)), d = __half22float2(*reinterpret_cast<const __half2*>(&v1));
    v[0] = c.x, v[1] = c.y, v[2] = d.x, v[3] = d.y;
}

// Exponent field of the scale of a block whose largest finite |entry| has the bits `top`: that
// entry is at most 1.75 times the top binade of the format, 2^(127 + exponents) in field units.
__device__ __forceinline__ uint32_t scale_field(uint32_t top, uint32_t exponents) {
    return min(max((top + 0x1fffffu) >> 23, 64u), 254u) - exponents;
}
__device__ __forceinline__ uint32_t finite_bits(float a) {
    const uint32_t u = __float_as_uint(a);
    return u < 0x7f800000u ? u : 0u;
}
// 32 random bits of an entry: 16 to round m with, 16 for v
__device__ __forceinline__ uint32_t random_bits(uint32_t x) {
    x = (x ^ (x >> 16)) * 0x7feb352du;
    return x ^ (x >> 15);
}
// The codes of m (with sign) and v: scaled by `inverse` and then by 2^-120 or 2^-112 an entry's fp32
// bits are the code followed by what is cut off, 20 or 21 bits, to which 16 random ones are added.
// Infinities and NaN become NaN; a positive v at least the smallest code.
__device__ __forceinline__ uint32_t code_m(float m, float inverse, uint32_t x) {
    const uint32_t u = __float_as_uint(__fmul_rn(__fmul_rn(fabsf(m), inverse), 0x1p-120f));
    return min(((u >> 4) + (x & 0xffffu)) >> 16, 0x7fu) | ((__float_as_uint(m) >> 24) & 0x80u);
}
__device__ __forceinline__ uint32_t code_v(float v, float inverse, uint32_t x) {
    const uint32_t u = __float_as_uint(__fmul_rn(__fmul_rn(v, inverse), 0x1p-112f));
    return max(min(((u >> 5) + (x >> 16)) >> 16, 0x7fu), v > 0.f ? 1u : 0u);
}
__device__ __forceinline__ float inverse_of(uint32_t field) { return __uint_as_float((254u - field) << 23); }

// The codes of a lane's eight entries where a moment is not finite, a v is zero, or a factor is not a
// normal number. Out of line: it would double the code that every block runs through.
__device__ __noinline__ void rare_codes(const float* m, const float* v, float m_inv, float v_inv, uint32_t x0, uint32_t* out) {
    for (int i = 0; i < 8; ++i) {
        const uint32_t x = random_bits(x0 + uint32_t((i >> 2) * 128 + (i & 3)) * 0x9e3779b1u);
        const int at = 8 * (i & 3);
        if (at == 0) out[i >> 2] = out[2 + (i >> 2)] = 0;
        out[i >> 2] |= code_m(m[i], m_inv, x) << at;
        out[2 + (i >> 2)] |= code_v(v[i], v_inv, x) << at;
    }
}
__device__ __noinline__ void finite_tops(const float* m, const float* v, uint32_t* tops) {
    tops[0] = tops[1] = 0;
    for (int i = 0; i < 8; ++i) {
        tops[0] = max(tops[0], finite_bits(fabsf(m[i])));
        tops[1] = max(tops[1], finite_bits(v[i]));
    }
}

// 256 neighbouring entries of a tensor with 8-bit moments, by a warp, four neighbouring ones of a lane
// at a time. A Stage is where their operands arrive in shared memory; every lane copies what it
// will read itself, so that its own wait is all that the copies need.
template <class TG>
struct Stage {
    float4 p[2][32];
    typename Raw4<TG>::type g[2][32];
    uint32_t m[2][32], v[2][32];

    __device__ __forceinline__ void fetch(const float* gp, const TG* gg, const uint8_t* gm, const uint8_t* gv) {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int e = j * 128 + lane * 4;
            copy_async<16>(&p[j][lane], gp + e);
            copy_async<4 * sizeof(TG)>(&g[j][lane], gg + e);
            copy_async<4>(&m[j][lane], gm + e);
            copy_async<4>(&v[j][lane], gv + e);
        }
    }
};
template <class TG>
struct Block8 {
    // the exponent fields of the new scales come back in m_field and v_field
    static __device__ __forceinline__ void step(const Stage<TG>& in, float m_scale, float v_scale, float* at_p,
                                                __nv_bfloat16* at_copy, int64_t s, float2 keep, const AdamwState& st,
                                                const AdamwRates& r, float clip, uint32_t& m_field, uint32_t& v_field) {
        const int lane = threadIdx.x & 31;
        // m_scale is a power of two: code (m_scale beta1) is (code m_scale) beta1, bit for bit
        const float beta1 = m_scale * r.beta1, beta2 = v_scale * r.beta2;
        float mf[8], vf[8];
        float m_top = 0.f, v_top = 0.f;
        bool zero = false;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int e = j * 128 + lane * 4;
            float gf[4], pf[4], m4[4], v4[4];
            unpack(in.g[j][lane], gf);
            unpack(in.p[j][lane], pf);
            from_codes(in.m[j][lane], in.v[j][lane], m4, v4);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                moments(__fmul_rn(gf[k], clip), m4[k], v4[k], beta1, beta2, r);
                m_top = max_or_nan(m_top, fabsf(m4[k]));
                v_top = max_or_nan(v_top, v4[k]);
                zero |= v4[k] == 0.f;
                pf[k] = update(pf[k], m4[k], v4[k], keep, r);
                mf[j * 4 + k] = m4[k];
                vf[j * 4 + k] = v4[k];
            }
            *reinterpret_cast<float4*>(at_p + e) = make_float4(pf[0], pf[1], pf[2], pf[3]);
            if (at_copy) *reinterpret_cast<uint2*>(at_copy + e) = make_uint2(pair(pf[0], pf[1]), pair(pf[2], pf[3]));
        }
        // the bits of a NaN or an infinity are above those of every finite number
        uint32_t m_bits = __reduce_max_sync(0xffffffffu, __float_as_uint(m_top) & 0x7fffffffu);
        uint32_t v_bits = __reduce_max_sync(0xffffffffu, __float_as_uint(v_top) & 0x7fffffffu);
        const bool odd = max(m_bits, v_bits) >= 0x7f800000u;
        if (odd) {
            float m8[8], v8[8];
            uint32_t tops[2];
#pragma unroll
            for (int i = 0; i < 8; ++i) m8[i] = mf[i], v8[i] = vf[i];
            finite_tops(m8, v8, tops);
            m_bits = __reduce_max_sync(0xffffffffu, tops[0]);
            v_bits = __reduce_max_sync(0xffffffffu, tops[1]);
        }
        m_field = scale_field(m_bits, 8);
        v_field = scale_field(v_bits, 15);
        const float m_inv = inverse_of(m_field), v_inv = inverse_of(v_field);
        const uint32_t x0 = uint32_t(s + lane * 4) * 0x9e3779b1u + r.key;
        uint32_t codes[4];   // of m, then of v
        if (!odd && m_field <= 133u && v_field <= 141u && !__any_sync(0xffffffffu, zero)) {
            // All finite, no v zero, and both factors of an entry in one normal number: the codes are
            // byte 2 of a sum each, gathered four at a time; a v below the smallest code is raised to it,
            // which rounds to that code whatever the random bits.
            const float m_low = m_inv * 0x1p-120f, v_low = v_inv * 0x1p-112f;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                uint32_t ms[4], vs[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t x = random_bits(x0 + uint32_t(j * 128 + k) * 0x9e3779b1u);
                    ms[k] = (__float_as_uint(__fmul_rn(fabsf(mf[j * 4 + k]), m_low)) >> 4) + (x & 0xffffu);
                    vs[k] = (__float_as_uint(fmaxf(__fmul_rn(vf[j * 4 + k], v_low), 0x1p-128f)) >> 5) + (x >> 16);
                }
                const uint32_t s01 = __byte_perm(__float_as_uint(mf[j * 4]), __float_as_uint(mf[j * 4 + 1]), 0x73);
                const uint32_t s23 = __byte_perm(__float_as_uint(mf[j * 4 + 2]), __float_as_uint(mf[j * 4 + 3]), 0x73);
                codes[j] = __byte_perm(__byte_perm(ms[0], ms[1], 0x62), __byte_perm(ms[2], ms[3], 0x62), 0x5410) |
                           (__byte_perm(s01, s23, 0x5410) & 0x80808080u);
                codes[2 + j] = __byte_perm(__byte_perm(vs[0], vs[1], 0x62), __byte_perm(vs[2], vs[3], 0x62), 0x5410);
            }
        } else {
            float m8[8], v8[8];
            uint32_t c4[4];
#pragma unroll
            for (int i = 0; i < 8; ++i) m8[i] = mf[i], v8[i] = vf[i];
            rare_codes(m8, v8, m_inv, v_inv, x0, c4);
#pragma unroll
            for (int i = 0; i < 4; ++i) codes[i] = c4[i];
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int e = j * 128 + lane * 4;
            *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(st.m) + s + e) = codes[j];
            *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(st.v) + s + e) = codes[2 + j];
        }
    }
};

// The same for a tensor's last, shorter block and for tensors without vector alignment: entry by entry.
template <class TG>
__device__ __noinline__ void ragged_block8(const AdamwTensor& a, const TG* g, const AdamwState& st, const AdamwRates& r,
                                           int64_t at, float clip, float2 keep) {
    const int64_t s = a.start + at;
    const int lane = threadIdx.x & 31;
    const float m_scale = st.m_scale[s / kAdamwBlock], v_scale = st.v_scale[s / kAdamwBlock];
    uint8_t* ms = static_cast<uint8_t*>(st.m) + s;
    uint8_t* vs = static_cast<uint8_t*>(st.v) + s;
    float m[8], v[8];
    uint32_t m_top = 0, v_top = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int e = lane + 32 * j;
        m[j] = v[j] = 0.f;
        if (at + e >= a.numel) continue;
        float m4[4], v4[4];
        from_codes(ms[e], vs[e], m4, v4);
        m[j] = __fmul_rn(m4[0], m_scale);
        v[j] = __fmul_rn(v4[0], v_scale);
        moments(__fmul_rn(load_f(g + at + e), clip), m[j], v[j], r.beta1, r.beta2, r);
        m_top = max(m_top, finite_bits(fabsf(m[j])));
        v_top = max(v_top, finite_bits(v[j]));
        const float p = update(a.p[at + e], m[j], v[j], keep, r);
        a.p[at + e] = p;
        if (a.copy) a.copy[at + e] = __float2bfloat16_rn(p);
    }
    const uint32_t m_field = scale_field(__reduce_max_sync(0xffffffffu, m_top), 8);
    const uint32_t v_field = scale_field(__reduce_max_sync(0xffffffffu, v_top), 15);
    if (lane == 0) {
        st.m_scale[s / kAdamwBlock] = __uint_as_float(m_field << 23);
        st.v_scale[s / kAdamwBlock] = __uint_as_float(v_field << 23);
    }
    const float m_inv = inverse_of(m_field), v_inv = inverse_of(v_field);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int e = lane + 32 * j;
        const uint32_t x = random_bits(uint32_t(s + e) * 0x9e3779b1u + r.key);
        ms[e] = uint8_t(code_m(m[j], m_inv, x));
        vs[e] = uint8_t(code_v(v[j], v_inv, x));
    }
}

// a chunk with 32-bit moments
template <class TG>
__device__ __forceinline__ void chunk32(const AdamwTensor& a, const TG* g, const AdamwState& st, const AdamwRates& r,
                                        int64_t at, int n, bool vectors, float clip, float2 keep) {
    constexpr int V = kAdamwChunk / kThreads / 4;
    float* m = static_cast<float*>(st.m) + a.start + at;
    float* v = static_cast<float*>(st.v) + a.start + at;
    float* p = a.p + at;
    __nv_bfloat16* copy = a.copy ? a.copy + at : nullptr;
    g += at;
    int done = 0;
    if (vectors) {
        done = n & ~3;
        float4 rp[V], rm[V], rv[V];
        typename Raw4<TG>::type rg[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int i = (j * kThreads + int(threadIdx.x)) * 4;
            if (i >= done) continue;
            rp[j] = *reinterpret_cast<const float4*>(p + i);
            rg[j] = __ldcs(reinterpret_cast<const typename Raw4<TG>::type*>(g + i));
            rm[j] = *reinterpret_cast<const float4*>(m + i);
            rv[j] = *reinterpret_cast<const float4*>(v + i);
        }
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int i = (j * kThreads + int(threadIdx.x)) * 4;
            if (i >= done) continue;
            float pf[4], gf[4], mf[4], vf[4];
            unpack(rp[j], pf);
            unpack(rg[j], gf);
            unpack(rm[j], mf);
            unpack(rv[j], vf);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                moments(__fmul_rn(gf[k], clip), mf[k], vf[k], r.beta1, r.beta2, r);
                pf[k] = update(pf[k], mf[k], vf[k], keep, r);
            }
            *reinterpret_cast<float4*>(p + i) = make_float4(pf[0], pf[1], pf[2], pf[3]);
            *reinterpret_cast<float4*>(m + i) = make_float4(mf[0], mf[1], mf[2], mf[3]);
            *reinterpret_cast<float4*>(v + i) = make_float4(vf[0], vf[1], vf[2], vf[3]);
            if (copy) *reinterpret_cast<uint2*>(copy + i) = make_uint2(pair(pf[0], pf[1]), pair(pf[2], pf[3]));
        }
    }
    for (int i = done + int(threadIdx.x); i < n; i += kThreads) {
        float mf = m[i], vf = v[i];
        moments(__fmul_rn(load_f(g + i), clip), mf, vf, r.beta1, r.beta2, r);
        const float pf = update(p[i], mf, vf, keep, r);
        p[i] = pf;
        m[i] = mf;
        v[i] = vf;
        if (copy) copy[i] = __float2bfloat16_rn(pf);
    }
}

// blocks of a warp whose operands are on their way or being used
constexpr int kStages = 3;
template <class TG, int BITS>
constexpr int kSmem = BITS == 8 ? int(sizeof(Stage<TG>)) * kStages * (kThreads / 32) : 0;

template <class TG, int BITS>
__global__ void __launch_bounds__(kThreads, BITS == 8 ? 3 : 2)
    adamw_kernel(const AdamwTensor* __restrict__ tensors, const int32_t* __restrict__ chunk_tensor, int tensor0,
                 int chunk0, int chunks, const __grid_constant__ Gradients grads,
                 const __grid_constant__ AdamwState st, const __grid_constant__ AdamwRates r,
                 const float2* __restrict__ partial, int parts, float* __restrict__ norm_out) {
    float clip = 1.f;
    if (r.max_norm > 0.f) {
        __shared__ float2 smem[kThreads / 32];
        float2 sum = make_float2(0.f, 0.f);
        for (int i = threadIdx.x; i < parts; i += kThreads) sum = add(sum, partial[i]);
        sum = block_sum(sum, smem);
        const float norm = sqrtf(__fadd_rn(sum.x, sum.y));
        if (blockIdx.x == 0 && threadIdx.x == 0) *norm_out = norm;
        if (!(norm < __uint_as_float(0x7f800000u))) return;
        clip = fminf(r.max_norm / norm, 1.f);
    }
    stretches(tensors, chunk_tensor, chunk0, chunks, blockIdx.x, gridDim.x,
              [&](const AdamwTensor& a, int t, int64_t first, int64_t last) {
        const TG* g = static_cast<const TG*>(grads.g[t - tensor0]);
        if (g == nullptr) return;
        const float2 keep = keeps(r.lr, a.decay);
        const bool vectors = aligned4(g) && aligned4(a.p) && aligned4(a.copy);
        if constexpr (BITS == 32) {
            for (int64_t at = first; at < last; at += kAdamwChunk)
                chunk32(a, g, st, r, at, int(last - at < kAdamwChunk ? last - at : kAdamwChunk), vectors, clip, keep);
        } else {
            // A warp takes a run of neighbouring blocks, 32 at a time: lane k reads the scales of the k-th
            // and writes its new ones, all 32 together. (Scales read and written one by one, by warps that
            // take blocks in turn, share 32-byte sectors between a load of one warp and a store of
            // another: that alone cost 0.62 ms against 0.45 ms at 200M entries.)
            constexpr int kWarps = kThreads / 32;
            extern __shared__ float4 stage_memory[];
            const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
            Stage<TG>* stage = reinterpret_cast<Stage<TG>*>(stage_memory) + warp * kStages;
            const int64_t full = vectors ? (last - first) / kAdamwBlock : 0;
            const int64_t from = full * warp / kWarps, mine = full * (warp + 1) / kWarps - from;
            int64_t now = first + from * kAdamwBlock, at = now;   // of the block in hand, and of the one fetched next
            const uint8_t* sm = static_cast<const uint8_t*>(st.m) + a.start;
            const uint8_t* sv = static_cast<const uint8_t*>(st.v) + a.start;
            float* m_scales = st.m_scale + (a.start + now) / kAdamwBlock;
            float* v_scales = st.v_scale + (a.start + now) / kAdamwBlock;
            int put = 0, get = 0;
            const auto fetch = [&](int64_t k) {
                if (k < mine) stage[put].fetch(a.p + at, g + at, sm + at, sv + at);
                copies_commit();
                at += kAdamwBlock;
                put = put + 1 == kStages ? 0 : put + 1;
            };
#pragma unroll
            for (int k = 0; k < kStages - 1; ++k) fetch(k);
#pragma unroll 1
            for (int64_t k0 = 0; k0 < mine; k0 += 32) {
                const int some = int(mine - k0 < 32 ? mine - k0 : 32);
                float ms = lane < some ? m_scales[k0 + lane] : 0.f, vs = lane < some ? v_scales[k0 + lane] : 0.f;
#pragma unroll 1
                for (int k = 0; k < some; ++k) {
                    fetch(k0 + k + kStages - 1);
                    const float m_scale = __shfl_sync(0xffffffffu, ms, k), v_scale = __shfl_sync(0xffffffffu, vs, k);
                    uint32_t m_field, v_field;
                    copies_wait<kStages - 1>();
                    Block8<TG>::step(stage[get], m_scale, v_scale, a.p + now, a.copy ? a.copy + now : nullptr,
                                     a.start + now, keep, st, r, clip, m_field, v_field);
                    if (lane == k) ms = __uint_as_float(m_field << 23), vs = __uint_as_float(v_field << 23);
                    now += kAdamwBlock;
                    get = get + 1 == kStages ? 0 : get + 1;
                }
                if (lane < some) m_scales[k0 + lane] = ms, v_scales[k0 + lane] = vs;
            }
            copies_wait<0>();
            for (int64_t b = full + (warp - full % kWarps + kWarps) % kWarps; first + b * kAdamwBlock < last; b += kWarps)
                ragged_block8(a, g, st, r, first + b * kAdamwBlock, clip, keep);
        }
    });
}

template <class TG, int BITS>
cudaError_t run(const AdamwTensor* tensors, const int32_t* chunk_tensor, const int32_t* first_chunk, int n_tensors,
                const void* const* grads, const AdamwState& st, const AdamwRates& r, float* norm_out, float2* partial,
                cudaStream_t s) {
    auto* k = adamw_kernel<TG, BITS>;
    constexpr int smem = kSmem<TG, BITS>;
    if constexpr (smem > 0) {
        static std::atomic<uint64_t> set{0};   // devices (by bit) whose limit is raised
        int dev = 0;
        cudaGetDevice(&dev);
        const uint64_t bit = uint64_t(1) << (dev & 63);
        if (!(set.load(std::memory_order_relaxed) & bit)) {
            const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
            if (e != cudaSuccess) return e;
            set.fetch_or(bit, std::memory_order_relaxed);
        }
    }
    Gradients g;
    const auto each = [&](auto&& launch) -> cudaError_t {
        for (int t0 = 0; t0 < n_tensors; t0 += kAdamwLaunch) {
            const int t1 = t0 + kAdamwLaunch < n_tensors ? t0 + kAdamwLaunch : n_tensors;
            const int chunks = first_chunk[t1] - first_chunk[t0];
            int runs = grid_for((const void*)k, kThreads, 1, chunks > 0 ? chunks : 1, smem);
            if (runs > kAdamwRuns) runs = kAdamwRuns;
            for (int t = t0; t < t1; ++t) g.g[t - t0] = grads[t];
            launch(t0, first_chunk[t0], chunks, runs);
            const cudaError_t e = cudaGetLastError();
            if (e != cudaSuccess) return e;
        }
        return cudaSuccess;
    };
    int parts = 0;
    if (r.max_norm > 0.f) {
        const cudaError_t e = each([&](int t0, int c0, int chunks, int runs) {
            adamw_norm_kernel<TG><<<runs * kNormSplit, kThreads, 0, s>>>(tensors, chunk_tensor, t0, c0, chunks, g, partial + parts);
            parts += runs * kNormSplit;
        });
        if (e != cudaSuccess) return e;
    }
    return each([&](int t0, int c0, int chunks, int runs) {
        k<<<runs, kThreads, smem, s>>>(tensors, chunk_tensor, t0, c0, chunks, g, st, r, partial, parts, norm_out);
    });
}

}  // namespace

size_t adamw_workspace_bytes(int n_tensors) {
    return size_t((n_tensors + kAdamwLaunch - 1) / kAdamwLaunch) * kAdamwRuns * kNormSplit * sizeof(float2);
}

cudaError_t adamw_step(const AdamwTensor* tensors, const int32_t* chunk_tensor, const int32_t* first_chunk_host,
                       int n_tensors, const void* const* grads, int g_bf16, const AdamwState& st,
                       const AdamwRates& r, float* norm_out, void* ws, cudaStream_t s) {
    float2* partial = static_cast<float2*>(ws);
    const auto go = [&](auto tg) {
        using TG = decltype(tg);
        return st.bits == 8 ? run<TG, 8>(tensors, chunk_tensor, first_chunk_host, n_tensors, grads, st, r, norm_out, partial, s)
                            : run<TG, 32>(tensors, chunk_tensor, first_chunk_host, n_tensors, grads, st, r, norm_out, partial, s);
    };
    return g_bf16 ? go(__nv_bfloat16{}) : go(0.f);
}

}  // namespace e3gb
