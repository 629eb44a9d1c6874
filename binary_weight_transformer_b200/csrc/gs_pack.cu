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
// cover the memory latency without unrolling.
#include "gs_internal.cuh"

namespace lowbit {
namespace {

constexpr int kThreads = 256;
constexpr int kUnit = 256;  // codes per warp

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
            const uint4 u0 = ld_act_u4(static_cast<const float *>(w) + at);
            const uint4 u1 = ld_act_u4(static_cast<const float *>(w) + at + 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[i] = __uint_as_float((&u0.x)[i]);
                v[4 + i] = __uint_as_float((&u1.x)[i]);
            }
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

template <bool BF16>
__global__ void __launch_bounds__(kThreads)
gs_pack_kernel(const void *__restrict__ w, int64_t N, int64_t K, int64_t ldw, int vec, int gshift, int64_t units,
               uint8_t *__restrict__ packed, int64_t ldp, void *__restrict__ s_g, int s_bf16, int64_t lds,
               int32_t *status)
{
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
    if (unit >= N * units) return;
    const int64_t n = unit / units;
    const int64_t k0 = (unit % units) * kUnit + lane * 8;
    const int64_t left = K - k0;
    const int valid = left >= 8 ? 8 : left > 0 ? static_cast<int>(left) : 0;

    float v[8];
    load8<BF16>(w, n * ldw + k0, valid, vec != 0, v);
    uint32_t top = 0;  // |w| as bits: non-finite values sort above finite ones
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
    const int lanes = (1 << gshift) >> 3;
    for (int o = 1; o < lanes; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (!finite_bits(top)) {
        if ((lane & (lanes - 1)) == 0) report(status, LOWBIT_ERR_NONFINITE);
    }
    float s = __fdiv_rn(__uint_as_float(top), 7.0f);
    const __nv_bfloat16 sb = __float2bfloat16_rn(s);
    if (s_bf16) s = __bfloat162float(sb);
    if ((lane & (lanes - 1)) == 0 && k0 < K) {
        const int64_t at = n * lds + (k0 >> gshift);
        if (s_bf16) static_cast<__nv_bfloat16 *>(s_g)[at] = sb;
        else static_cast<float *>(s_g)[at] = s;
    }

    uint32_t word = 0;
    if (s >= 0x1p-60f && s <= 0x1p+60f) {
        // u = RN(w * RN(1/s)) is within 7.03 * 2^-23 < 1e-6 of the exact
        // quotient, so both round to the same integer unless u is that near
        // a half; about one weight in 10^5 is, and goes by the definition.
        // The rounding is the addition of 1.5 * 2^23, whose low bits are then
        // the code in two's complement.  |u| <= 7.03: a bf16 scale is at most
        // 2^-8 below the quotient, so no clip.
        const float c = __frcp_rn(s);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float u = __fmul_rn(v[i], c);
            const float m = __fadd_rn(u, 12582912.0f);
            uint32_t code = __float_as_uint(m);
            if (fabsf(__fsub_rn(u, __fsub_rn(m, 12582912.0f))) > 0.49999f)
                code = static_cast<uint32_t>(code_exact(v[i], s));
            word |= (code & 15u) << (8 * (i & 3) + 4 * (i >> 2));
        }
    } else if (s > 0.0f) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            word |= (static_cast<uint32_t>(code_exact(v[i], s)) & 15u) << (8 * (i & 3) + 4 * (i >> 2));
    }
    if (k0 / 2 < ldp) *reinterpret_cast<uint32_t *>(packed + n * ldp + k0 / 2) = word;
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads)
gs_unpack_kernel(const uint8_t *__restrict__ packed, int64_t ldp, const void *__restrict__ s_g, int s_bf16,
                 int64_t lds, int64_t N, int64_t K, int gshift, int64_t words, void *__restrict__ w, int64_t ldw,
                 int vec, int32_t *status)
{
    pdl_wait();
    pdl_trigger();
    const int64_t idx = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    if (idx >= N * words) return;
    const int64_t n = idx / words;
    const int64_t wi = idx % words;
    const uint32_t word = ld_act_u32(packed + n * ldp + wi * 4);
    const int64_t k0 = wi * 8;
    const int64_t at = n * lds + (k0 >> gshift);
    const float s = s_bf16 ? __uint_as_float(static_cast<uint32_t>(
                                 ld_act_u16(static_cast<const uint16_t *>(s_g) + at)) << 16)
                           : ld_act_f32(static_cast<const float *>(s_g) + at);
    const int valid = K - k0 >= 8 ? 8 : static_cast<int>(K - k0);
    bool bad = false;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int bit = 8 * (i & 3) + 4 * (i >> 2);
        int c = static_cast<int>(word << (28 - bit)) >> 28;
        if (c == -8 || (i >= valid && c != 0)) {
            bad = true;
            c = 0;
        }
        v[i] = __fmul_rn(static_cast<float>(c), s);
    }
    if (bad) report(status, LOWBIT_ERR_RESERVED_CODE);
    if (valid == 8 && vec) {
        if constexpr (BF16) {
            uint4 u;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
                (&u.x)[i] = *reinterpret_cast<const uint32_t *>(&p);
            }
            *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(w) + n * ldw + k0) = u;
        } else {
            float4 *dst = reinterpret_cast<float4 *>(static_cast<float *>(w) + n * ldw + k0);
            dst[0] = make_float4(v[0], v[1], v[2], v[3]);
            dst[1] = make_float4(v[4], v[5], v[6], v[7]);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (i < valid) {
            if constexpr (BF16) static_cast<__nv_bfloat16 *>(w)[n * ldw + k0 + i] = __float2bfloat16_rn(v[i]);
            else static_cast<float *>(w)[n * ldw + k0 + i] = v[i];
        }
    }
}

bool rows_aligned(const void *p, int64_t ld, int64_t esz)
{
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (ld * esz) % 16 == 0;
}

}  // namespace

lowbit_status gs_pack_launch(const void *w, int w_bf16, int64_t N, int64_t K, int64_t ldw, int gshift, uint8_t *packed,
                             int64_t ldp, void *s_g, int s_bf16, int64_t lds, int32_t *status, cudaStream_t st)
{
    const int64_t units = (ldp * 2 + kUnit - 1) / kUnit;
    const int64_t blocks = (N * units + kThreads / 32 - 1) / (kThreads / 32);
    if (blocks > INT32_MAX) return LOWBIT_ERR_UNSUPPORTED;
    const int vec = rows_aligned(w, ldw, w_bf16 ? 2 : 4) ? 1 : 0;
    return launch_pdl(w_bf16 ? gs_pack_kernel<true> : gs_pack_kernel<false>, dim3(static_cast<unsigned>(blocks)),
                      dim3(kThreads), 0, st, 0, w, N, K, ldw, vec, gshift, units, packed, ldp, s_g, s_bf16, lds, status);
}

lowbit_status gs_unpack_launch(const uint8_t *packed, int64_t ldp, const void *s_g, int s_bf16, int64_t lds, int64_t N,
                               int64_t K, int gshift, void *w, int w_bf16, int64_t ldw, int32_t *status,
                               cudaStream_t st)
{
    const int64_t words = (K + 7) / 8;
    const int64_t blocks = (N * words + kThreads - 1) / kThreads;
    if (blocks > INT32_MAX) return LOWBIT_ERR_UNSUPPORTED;
    const int vec = rows_aligned(w, ldw, w_bf16 ? 2 : 4) ? 1 : 0;
    return launch_pdl(w_bf16 ? gs_unpack_kernel<true> : gs_unpack_kernel<false>, dim3(static_cast<unsigned>(blocks)),
                      dim3(kThreads), 0, st, 0, packed, ldp, s_g, s_bf16, lds, N, K, gshift, words, w, ldw, vec,
                      status);
}

}  // namespace lowbit
