// gs_pack.cu -- 4-bit weights with one scale per group: quantise, pack, and
// decode back to values.
//
//   s[n,g] = round_s(max_{k in g} |w[n,k]| / 7)     (fp32 quotient, then the scale's type)
//   c[n,k] = clip(rint(w[n,k] / s[n,g]), -7, 7)     the integer nearest to the exact
//            quotient, a half to the even one; s = 0 gives c = 0
//
// Both kernels move bytes: a warp takes 256 consecutive codes of a row, eight
// per lane, which is one packed word per lane, one 128-byte store per warp and
// whole groups (32 to 256 codes = 4 to 32 lanes) whose maximum is a few
// shuffles.  32 (fp32) or 16 (bf16) bytes per lane in flight at full occupancy
// cover the memory latency; what held the packer back was instructions (25 per
// weight at first: 64-bit divisions for the address, an IEEE division and
// reciprocal per lane).  A lane's eight fp32 values are
// one 32-byte access where rows allow it: as two of 16 bytes, every 32-byte
// sector crosses the L2 twice.
#include "gs_internal.cuh"

namespace lowbit {
namespace {

constexpr int kThreads = 256;
constexpr int kUnit = 256;  // codes per warp and piece
constexpr int kInFlight = 4;  // words per thread of a large unpack

// The code of one weight by the definition, whatever the scale's size.
// qf = RN(a / s) is monotone in the exact quotient and every half is a float,
// so qf lies on the right side of a half unless it equals one; there the
// residual a - qf * s (one rounding of an exact value: its sign is right)
// tells.  Small operands are scaled up first, exactly, so that the residual
// cannot underflow.
__device__ __noinline__ int code_exact(float w, float s)
{
    float a = fabsf(w);
    if (s < 0x1p-60f) {
        a *= 0x1p+80f;
        s *= 0x1p+80f;
    }
    const float qf = __fdiv_rn(a, s);
    float f = rintf(qf);
    if (fabsf(qf - truncf(qf)) == 0.5f) {
        const float r = __fmaf_rn(-qf, s, a);
        if (r > 0.0f) f = ceilf(qf);
        if (r < 0.0f) f = floorf(qf);
    }
    const int c = static_cast<int>(fminf(f, 7.0f));
    return w < 0.0f ? -c : c;
}

template <bool BF16>
__device__ __forceinline__ void load8(const void *w, int64_t at, int valid, bool vec, float (&v)[8])
{
    if (valid >= 8 && vec) {
        if constexpr (BF16) {
            const uint4 u = ld_act_u4(static_cast<const uint16_t *>(w) + at);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t x = (&u.x)[i >> 1];
                v[i] = __uint_as_float((i & 1) ? (x & 0xffff0000u) : (x << 16));
            }
        } else {
            asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                         : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
                         : "l"(static_cast<const float *>(w) + at) : "memory");
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (i < valid) {
            if constexpr (BF16)
                v[i] = __uint_as_float(static_cast<uint32_t>(ld_act_u16(static_cast<const uint16_t *>(w) + at + i)) << 16);
            else
                v[i] = ld_act_f32(static_cast<const float *>(w) + at + i);
        } else {
            v[i] = 0.0f;
        }
    }
}

// RN(a / 7).  Markstein's correction (IBM J. Res. Dev. 34, 1990): with y =
// RN(1/7) and q = RN(a y), the residual r = a - 7 q is exact in one fma and
// RN(q + r y) is the correctly rounded quotient, where nothing underflows.
__device__ __forceinline__ float seventh(float a)
{
    if (a < 0x1p-100f) return __fdiv_rn(a, 7.0f);
    constexpr float y = 1.0f / 7.0f;
    const float q = __fmul_rn(a, y);
    return __fmaf_rn(__fmaf_rn(-7.0f, q, a), y, q);
}

// The packed word of a lane's eight weights, and (from the first lane of each
// group of `lanes`) its scale.
template <bool S16, int lanes>
__device__ __forceinline__ uint32_t pack_word(const float (&v)[8], int lane, bool owns, void *s_at,
                                              int32_t *status)
{
    uint32_t top = 0;  // |w| as bits: non-finite values sort above finite ones
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
#pragma unroll
    for (int o = 1; o < lanes; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const bool first = (lane & (lanes - 1)) == 0;
    if (first && !finite_bits(top)) report(status, LOWBIT_ERR_NONFINITE);
    float s = seventh(__uint_as_float(top));
    if constexpr (S16) {
        const __nv_bfloat16 b = __float2bfloat16_rn(s);
        s = __bfloat162float(b);
        if (first && owns) *static_cast<__nv_bfloat16 *>(s_at) = b;
    } else {
        if (first && owns) *static_cast<float *>(s_at) = s;
    }
    if (s >= 0x1p-60f && s <= 0x1p+60f) {
        // u = RN(w * c), c within 2^-23 of 1/s (rcp.approx: 1 ulp), is within
        // 7.03 * 1.5 * 2^-23 < 1.3e-6 of the exact quotient, so both round to
        // the same integer unless u is that near a half; where one of eight
        // weights is within 1e-5 (one lane in 10^4), all go by the definition.
        // The rounding is the addition of 1.5 * 2^23, whose low bits are then
        // the code in two's complement.  |u| <= 7.03: a bf16 scale is at most
        // 2^-8 below the quotient, so no clip.
        float c;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(c) : "f"(s));
        float m[8], far = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float u = __fmul_rn(v[i], c);
            m[i] = __fadd_rn(u, 12582912.0f);
            far = fmaxf(far, fabsf(__fsub_rn(u, __fsub_rn(m[i], 12582912.0f))));
        }
        if (far > 0.49999f) {
#pragma unroll
            for (int i = 0; i < 8; ++i) m[i] = __int_as_float(code_exact(v[i], s));
        }
        // low bytes of four codes each, then their low nibbles side by side
        uint32_t four[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t a = __byte_perm(__float_as_uint(m[4 * h]), __float_as_uint(m[4 * h + 1]), 0x0040);
            const uint32_t b = __byte_perm(__float_as_uint(m[4 * h + 2]), __float_as_uint(m[4 * h + 3]), 0x0040);
            four[h] = __byte_perm(a, b, 0x5410);
        }
        return (four[0] & 0x0f0f0f0fu) | ((four[1] << 4) & 0xf0f0f0f0u);
    }
    uint32_t word = 0;
    if (s > 0.0f) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            word |= (static_cast<uint32_t>(code_exact(v[i], s)) & 15u) << (8 * (i & 3) + 4 * (i >> 2));
    }
    return word;
}

template <bool BF16, bool S16, int GS>
__global__ void __launch_bounds__(kThreads, 8)
gs_pack_kernel(const void *__restrict__ w, int64_t N, int64_t K, int64_t ldw, int vec, int64_t units,
               uint8_t *__restrict__ packed, int64_t ldp, uint8_t *__restrict__ s_g, int64_t lds, int32_t *status)
{
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    int64_t n, at;
    divide(static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5), units, n, at);
    if (n >= N) return;
    const int64_t k0 = at * kUnit + lane * 8;
    const int64_t left = K - k0;
    float v[8];
    load8<BF16>(w, n * ldw + k0, left >= 8 ? 8 : left > 0 ? static_cast<int>(left) : 0, vec != 0, v);
    const uint32_t word = pack_word<S16, (1 << GS) / 8>(v, lane, left > 0, s_g + (n * lds + (k0 >> GS)) * (S16 ? 2 : 4), status);
    if (k0 / 2 < ldp) *reinterpret_cast<uint32_t *>(packed + n * ldp + k0 / 2) = word;
}

template <bool BF16, int U>
__global__ void __launch_bounds__(kThreads)
gs_unpack_kernel(const uint8_t *__restrict__ packed, int64_t ldp, const void *__restrict__ s_g, int s_bf16,
                 int64_t lds, int64_t N, int64_t K, int gshift, int64_t words, void *__restrict__ w, int64_t ldw,
                 int vec, int32_t *status)
{
    pdl_wait();
    pdl_trigger();
    uint32_t word[U], scale[U];
    int64_t row[U], k0s[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t idx = (static_cast<int64_t>(blockIdx.x) * U + u) * kThreads + threadIdx.x;
        int64_t wi;
        divide(idx, words, row[u], wi);
        k0s[u] = wi * 8;
        word[u] = scale[u] = 0;
        if (row[u] < N) {
            word[u] = ld_act_u32(packed + row[u] * ldp + wi * 4);
            const int64_t at = row[u] * lds + (k0s[u] >> gshift);
            if (s_bf16) scale[u] = ld_act_u16(static_cast<const uint16_t *>(s_g) + at);
            else scale[u] = ld_act_u32(static_cast<const float *>(s_g) + at);
        }
    }
    bool bad = false;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (row[u] >= N) break;
        const float s = __uint_as_float(s_bf16 ? scale[u] << 16 : scale[u]);
        const int64_t n = row[u], k0 = k0s[u];
        const int valid = K - k0 >= 8 ? 8 : static_cast<int>(K - k0);
        // bits no code of the row owns, and reserved fields: a nibble 1000 is a
        // zero nibble of x, which the subtraction's borrow marks
        uint32_t codes = word[u];
        const uint32_t x = codes ^ 0x88888888u;
        if (((x - 0x11111111u) & ~x & 0x88888888u) != 0u || valid < 8) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t field = 15u << (8 * (i & 3) + 4 * (i >> 2));
                if ((codes & field) == (field & 0x88888888u) || (i >= valid && (codes & field) != 0u)) {
                    bad = true;
                    codes &= ~field;
                }
            }
        }
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = __fmul_rn(static_cast<float>(static_cast<int>(codes << (28 - 8 * (i & 3) - 4 * (i >> 2))) >> 28), s);
        if (valid == 8 && vec) {
            if constexpr (BF16) {
                uint4 o;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
                    (&o.x)[i] = *reinterpret_cast<const uint32_t *>(&p);
                }
                *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(w) + n * ldw + k0) = o;
            } else {
                asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                             ::"l"(static_cast<float *>(w) + n * ldw + k0), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]),
                               "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]) : "memory");
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (i < valid) {
                    if constexpr (BF16) static_cast<__nv_bfloat16 *>(w)[n * ldw + k0 + i] = __float2bfloat16_rn(v[i]);
                    else static_cast<float *>(w)[n * ldw + k0 + i] = v[i];
                }
            }
        }
    }
    if (bad) report(status, LOWBIT_ERR_RESERVED_CODE);
}

// Rows on which eight values are one aligned access.
bool rows_aligned(const void *p, int64_t ld, int64_t esz)
{
    return reinterpret_cast<uintptr_t>(p) % (8 * esz) == 0 && ld % 8 == 0;
}

struct PackArgs {
    const void *w;
    int64_t N, K, ldw;
    int vec;
    int64_t units;
    uint8_t *packed;
    int64_t ldp;
    uint8_t *s_g;
    int64_t lds;
    int32_t *status;
    unsigned blocks;
    cudaStream_t st;
};

template <bool BF16, bool S16, int GS>
lowbit_status pack_one(const PackArgs &a)
{
    return launch_pdl(gs_pack_kernel<BF16, S16, GS>, dim3(a.blocks), dim3(kThreads), 0, a.st, 0, a.w, a.N, a.K, a.ldw,
                      a.vec, a.units, a.packed, a.ldp, a.s_g, a.lds, a.status);
}

template <bool BF16, bool S16>
lowbit_status pack_groups(const PackArgs &a, int gshift)
{
    switch (gshift) {
    case 5: return pack_one<BF16, S16, 5>(a);
    case 6: return pack_one<BF16, S16, 6>(a);
    case 7: return pack_one<BF16, S16, 7>(a);
    default: return pack_one<BF16, S16, 8>(a);
    }
}

}  // namespace

lowbit_status gs_pack_launch(const void *w, int w_bf16, int64_t N, int64_t K, int64_t ldw, int gshift, uint8_t *packed,
                             int64_t ldp, void *s_g, int s_bf16, int64_t lds, int32_t *status, cudaStream_t st)
{
    const int64_t units = (ldp * 2 + kUnit - 1) / kUnit;
    const int64_t blocks = (N * units + kThreads / 32 - 1) / (kThreads / 32);
    if (blocks > INT32_MAX) return LOWBIT_ERR_UNSUPPORTED;
    const PackArgs a = {w, N, K, ldw, rows_aligned(w, ldw, w_bf16 ? 2 : 4) ? 1 : 0, units, packed, ldp,
                        static_cast<uint8_t *>(s_g), lds, status, static_cast<unsigned>(blocks), st};
    return w_bf16 ? (s_bf16 ? pack_groups<true, true>(a, gshift) : pack_groups<true, false>(a, gshift))
                  : (s_bf16 ? pack_groups<false, true>(a, gshift) : pack_groups<false, false>(a, gshift));
}

lowbit_status gs_unpack_launch(const uint8_t *packed, int64_t ldp, const void *s_g, int s_bf16, int64_t lds, int64_t N,
                               int64_t K, int gshift, void *w, int w_bf16, int64_t ldw, int32_t *status,
                               cudaStream_t st)
{
    const int64_t words = (K + 7) / 8;
    // several words per thread once that still fills the GPU
    const bool many = N * words >= static_cast<int64_t>(device_sm_count()) * 2048 * kInFlight;
    const int64_t per_block = kThreads * (many ? kInFlight : 1);
    const int64_t blocks = (N * words + per_block - 1) / per_block;
    if (blocks > INT32_MAX) return LOWBIT_ERR_UNSUPPORTED;
    const int vec = rows_aligned(w, ldw, w_bf16 ? 2 : 4) ? 1 : 0;
    auto kernel = w_bf16 ? (many ? gs_unpack_kernel<true, kInFlight> : gs_unpack_kernel<true, 1>)
                         : (many ? gs_unpack_kernel<false, kInFlight> : gs_unpack_kernel<false, 1>);
    return launch_pdl(kernel, dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0, st, 0, packed, ldp, s_g, s_bf16, lds,
                      N, K, gshift, words, w, ldw, vec, status);
}

}  // namespace lowbit
