// gs_mma.cu -- the group-scaled 4-bit product for few tokens, on the
// warp-level tensor-core instruction mma.sync m16n8k32 (s8 x s8 -> s32).
//
//   y[t,n] = s_x[t] * sum_g s_g[n,g] * (sum_{k in g} q[t,k] c[n,k])
//
// The inner sums are exact int32; the sum over groups is fp32.  The codes
// enter the integer sum as c << 4 (expanding a nibble to the top of its byte
// makes the sign free) and the factor 16 leaves in the last multiply, exactly.
//
// A = 16 tokens x 32 codes, B = 32 codes x 8 weight rows, C = 16 x 8.  The 32
// positions of a K step may be any 32 codes as long as A and B agree, so lane
// (g, t) of a warp loads ONE 16-byte piece of weight row g -- 32 consecutive
// codes, piece t of a unit of 128 -- and uses its words as the B fragments of
// the unit's four steps; every weight byte is loaded once, by one lane.  With
// groups of 128 the whole unit has one scale, and with 256 a warp takes two
// consecutive units and carries the integer sum.  With groups of 64 or 32
// a step may only hold codes of one group: the four lanes of a row exchange
// words (2 or 4 shuffles per 16 bytes) so that steps and groups line up.
//
// A block owns 8*R weight rows; its warps (and, in a cluster, its peers) split
// K by units, and the fp32 partial tiles are added in a fixed order.
#include "gs_internal.cuh"
#include "tc_common.cuh"

namespace lowbit {
namespace gsm {

constexpr int kUnit = 128;     // codes of a row per warp step
constexpr int kMaxWarps = 16;
constexpr int kMaxSplit = 4;   // blocks of a cluster

enum { kG128 = 0, kG64 = 1, kG32 = 2, kG256 = 3 };

__device__ __forceinline__ void mma_s8(int32_t (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                       uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The low `valid` bytes of a little-endian word.
__device__ __forceinline__ uint32_t keep_bytes(uint32_t v, int64_t valid)
{
    return valid >= 4 ? v : valid <= 0 ? 0u : v & ((1u << (8 * valid)) - 1u);
}

// Token codes k .. k+15 (k a multiple of 16) and k .. k+7, zero past K.  Rows
// are readable up to the next multiple of 16 codes.
__device__ __forceinline__ uint4 q16(const int8_t *row, int64_t k, int64_t K)
{
    if (row == nullptr || k >= K) return make_uint4(0, 0, 0, 0);
    uint4 v = ld_act_ca_u4(row + k);
    if (k + 16 > K) {
        v.x = keep_bytes(v.x, K - k);
        v.y = keep_bytes(v.y, K - k - 4);
        v.z = keep_bytes(v.z, K - k - 8);
        v.w = keep_bytes(v.w, K - k - 12);
    }
    return v;
}

__device__ __forceinline__ uint2 q8(const int8_t *row, int64_t k, int64_t K)
{
    if (row == nullptr || k >= K) return make_uint2(0, 0);
    uint2 v;
    asm volatile("ld.global.ca.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(row + k) : "memory");
    v.x = keep_bytes(v.x, K - k);
    v.y = keep_bytes(v.y, K - k - 4);
    return v;
}

// The token fragment words of a unit for one token row: step j uses q[2j]
// (the four codes of the word's low nibbles) and q[2j+1] (the high ones).
template <int GM>
__device__ __forceinline__ void load_tokens(const int8_t *row, int64_t k0, int64_t K, int t, uint32_t (&q)[8])
{
    if constexpr (GM == kG32) {
        // step j: word t of piece j
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint2 v = q8(row, k0 + 32 * j + 8 * t, K);
            q[2 * j] = v.x;
            q[2 * j + 1] = v.y;
        }
    } else {
        // steps 0,1 and 2,3: two consecutive words each
        const int64_t a = GM == kG128 || GM == kG256 ? 32 * t : t < 2 ? 32 * t : 32 * (t - 2) + 16;
        const int64_t b = GM == kG128 || GM == kG256 ? 32 * t + 16 : t < 2 ? 32 * (t + 2) : 32 * t + 16;
        const uint4 u = q16(row, k0 + a, K), v = q16(row, k0 + b, K);
        q[0] = u.x, q[1] = u.y, q[2] = u.z, q[3] = u.w;
        q[4] = v.x, q[5] = v.y, q[6] = v.z, q[7] = v.w;
    }
}

// The four lanes of a weight row hold its pieces 0..3; afterwards w[j] is the
// word the lane feeds to step j.
template <int GM>
__device__ __forceinline__ void line_up(uint4 &w, int t)
{
    if constexpr (GM == kG128 || GM == kG256) return;
    // the 2 x 2 blocks of the 4 x 4 word matrix (lane, word) change places
    const bool low = t < 2;
    const uint32_t r0 = __shfl_xor_sync(0xffffffffu, low ? w.z : w.x, 2);
    const uint32_t r1 = __shfl_xor_sync(0xffffffffu, low ? w.w : w.y, 2);
    const uint4 a = low ? make_uint4(w.x, w.y, r0, r1) : make_uint4(r0, r1, w.z, w.w);
    if constexpr (GM == kG64) {
        w = a;
        return;
    }
    const bool even = (t & 1) == 0;
    const uint32_t s0 = __shfl_xor_sync(0xffffffffu, even ? a.y : a.x, 1);
    const uint32_t s1 = __shfl_xor_sync(0xffffffffu, even ? a.w : a.z, 1);
    w = even ? make_uint4(a.x, s0, a.z, s1) : make_uint4(s0, a.y, s1, a.w);
}

// TOK: tokens per pass (8, 16 or 32); R: slabs of 8 weight rows.
template <int TOK, int GM, int R>
__global__ void __launch_bounds__(kMaxWarps * 32)
gs_mma_kernel(const GsArgs a, int64_t units, int split)
{
    constexpr int MT = TOK == 32 ? 2 : 1;        // 16-token tiles
    constexpr int EL = TOK == 8 ? 2 : 4;         // C elements in use
    constexpr int UN = TOK == 32 ? 2 : 4;        // units in flight
    constexpr int kElems = MT * R * EL;          // partial sums per lane
    constexpr int kRun = GM == kG256 ? 2 : 1;    // consecutive units of one warp
    extern __shared__ float red[];               // [warps][kElems][32], then [split - 1][kElems * 32]
    const int warps = blockDim.x >> 5;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    const int rank = split > 1 ? static_cast<int>(tc::cluster_rank()) : 0;
    const int64_t n0 = static_cast<int64_t>(blockIdx.x / split) * (8 * R);
    const int64_t groups = ((a.K - 1) >> a.gshift) + 1;
    const int64_t chunks = (a.K + 31) >> 5;      // 16-byte pieces of a row
    const bool experts = a.offsets != nullptr;

    bool waited = a.prefetch == 0;
    if (waited) pdl_wait();
    pdl_trigger();
    int64_t lo = 0, hi = a.M, step = TOK;
    const uint8_t *packed = a.packed;
    int64_t s_at = 0;
    if (experts) {
        gs_expert_rows(a.offsets, blockIdx.y, a.M, lo, hi, a.status);
        packed += blockIdx.y * a.pstride;
        s_at = blockIdx.y * a.sstride;
    } else {
        lo = static_cast<int64_t>(blockIdx.y) * TOK;
        step = static_cast<int64_t>(gridDim.y) * TOK;
    }

    for (int64_t tok = lo; tok < hi; tok += step) {
        const int8_t *row[MT][2];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int64_t r = tok + 16 * m + 8 * h + g;
                row[m][h] = r < hi && (TOK > 8 || h == 0) ? a.q + r * a.ldq : nullptr;
            }
        float acc[MT][R][EL];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int i = 0; i < EL; ++i) acc[m][r][i] = 0.0f;

        const int stride = warps * split * kRun;
        for (int64_t u0 = (rank * warps + warp) * kRun; u0 < units; u0 += static_cast<int64_t>(stride) * (UN / kRun)) {
            uint4 w[UN][R];
            float sc[UN][R];
#pragma unroll
            for (int i = 0; i < UN; ++i) {
                const int64_t u = u0 + static_cast<int64_t>(i / kRun) * stride + i % kRun;
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const int64_t n = n0 + 8 * r + g;
                    const int64_t c = 4 * u + t;
                    const int64_t grp = (c << 5) >> a.gshift;  // the scale this lane fetches for its row
                    w[i][r] = n < a.N && c < chunks ? ld_stream_u4(packed + n * a.ldp + c * 16) : make_uint4(0, 0, 0, 0);
                    sc[i][r] = n < a.N && grp < groups ? gs_scale(a.s_g, s_at + n * a.lds + grp, a.s_bf16) : 0.0f;
                }
            }
            if (!waited) {
                pdl_wait();
                waited = true;
            }
            int32_t c[MT][R][4];
#pragma unroll
            for (int i = 0; i < UN; ++i) {
                // a second unit past the end of the row is all zeros
                const int64_t u = u0 + static_cast<int64_t>(i / kRun) * stride + i % kRun;
                if (u - i % kRun >= units) break;
                uint32_t q[MT][2][8];
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    load_tokens<GM>(row[m][0], u * kUnit, a.K, t, q[m][0]);
                    if constexpr (TOK > 8) load_tokens<GM>(row[m][1], u * kUnit, a.K, t, q[m][1]);
                }
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    line_up<GM>(w[i][r], t);
                    constexpr int kGroups = GM == kG32 ? 4 : GM == kG64 ? 2 : 1;
                    constexpr int kSteps = 4 / kGroups;
#pragma unroll
                    for (int gr = 0; gr < kGroups; ++gr) {
                        // scales of the rows 2t and 2t+1 that this lane's C columns belong to
                        const float s0 = __shfl_sync(0xffffffffu, sc[i][r], 8 * t + kSteps * gr);
                        const float s1 = __shfl_sync(0xffffffffu, sc[i][r], 8 * t + 4 + kSteps * gr);
#pragma unroll
                        for (int m = 0; m < MT; ++m) {
                            if (i % kRun == 0) c[m][r][0] = c[m][r][1] = c[m][r][2] = c[m][r][3] = 0;
#pragma unroll
                            for (int s = 0; s < kSteps; ++s) {
                                const int j = gr * kSteps + s;
                                const uint32_t word = (&w[i][r].x)[j];
                                mma_s8(c[m][r], q[m][0][2 * j], TOK > 8 ? q[m][1][2 * j] : 0u, q[m][0][2 * j + 1],
                                       TOK > 8 ? q[m][1][2 * j + 1] : 0u, i4_expand(word, 0), i4_expand(word, 1));
                            }
                            if (i % kRun == kRun - 1) {
#pragma unroll
                                for (int x = 0; x < EL; ++x)
                                    acc[m][r][x] = __fmaf_rn(x & 1 ? s1 : s0, __int2float_rn(c[m][r][x]), acc[m][r][x]);
                            }
                        }
                    }
                }
            }
        }
        if (!waited) {
            pdl_wait();
            waited = true;
        }

#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int i = 0; i < EL; ++i) red[(warp * kElems + (m * R + r) * EL + i) * 32 + lane] = acc[m][r][i];
        __syncthreads();
        float *peers = red + warps * kElems * 32;
        if (split > 1 && rank > 0) {
            for (int idx = threadIdx.x; idx < kElems * 32; idx += blockDim.x) {
                float v = 0.0f;
                for (int w = 0; w < warps; ++w) v += red[w * kElems * 32 + idx];
                const uint32_t dst = tc::map_to_peer(tc::smem_u32(peers + (rank - 1) * kElems * 32 + idx), 0);
                asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(dst), "f"(v) : "memory");
            }
        }
        if (split > 1) tc::cluster_sync_all();
        if (rank == 0) {
            for (int idx = threadIdx.x; idx < kElems * 32; idx += blockDim.x) {
                float v = 0.0f;
                for (int w = 0; w < warps; ++w) v += red[w * kElems * 32 + idx];
                for (int p = 1; p < split; ++p) v += peers[(p - 1) * kElems * 32 + idx];
                const int e = idx >> 5, ln = idx & 31;
                const int m = e / (R * EL), r = e / EL % R, x = e % EL;
                const int64_t token = tok + 16 * m + (ln >> 2) + 8 * (x >> 1);
                const int64_t n = n0 + 8 * r + 2 * (ln & 3) + (x & 1);
                if (token < hi && n < a.N) {
                    // v carries the factor 16 of the shifted codes
                    const float f = __fmul_rn(v, __fmul_rn(ld_act_f32(a.s_x + token), 0.0625f));
                    if (a.y_bf16) static_cast<__nv_bfloat16 *>(a.y)[token * a.ldy + n] = __float2bfloat16_rn(f);
                    else static_cast<float *>(a.y)[token * a.ldy + n] = f;
                }
            }
        }
        if (split > 1) tc::cluster_sync_all();
        else __syncthreads();
    }
    if (!waited) pdl_wait();
}

template <int TOK, int GM, int R>
lowbit_status launch(const GsArgs &a, cudaStream_t st)
{
    constexpr int kElems = (TOK == 32 ? 2 : 1) * R * (TOK == 8 ? 2 : 4);
    const int64_t units = (a.K + kUnit - 1) / kUnit;
    const int64_t slabs = (a.N + 8 * R - 1) / (8 * R);
    int64_t ytiles, active;
    if (a.offsets != nullptr) {
        ytiles = a.E;
        active = a.E < a.M ? a.E : a.M;
    } else {
        ytiles = (a.M + TOK - 1) / TOK;
        if (ytiles > 65535) ytiles = 65535;
        active = ytiles;
    }
    // Warps per slab: enough for about 32 on every SM, at most one per
    // unit (pair of units).
    const int64_t want = static_cast<int64_t>(device_sm_count()) * 32;
    int64_t warps = 1, split = 1;
    const int64_t runs = GM == kG256 ? (units + 1) / 2 : units;
    while (warps < 8 && slabs * active * warps < want && warps * 2 <= runs) warps *= 2;
    while (split < kMaxSplit && slabs * active * warps * split < want && warps * split * 2 <= runs) split *= 2;
    if (slabs * split > INT32_MAX) return LOWBIT_ERR_UNSUPPORTED;
    const size_t smem = static_cast<size_t>(warps + split - 1) * kElems * 32 * 4;
    return launch_pdl(gs_mma_kernel<TOK, GM, R>, dim3(static_cast<unsigned>(slabs * split), static_cast<unsigned>(ytiles)),
                      dim3(static_cast<unsigned>(warps * 32)), smem, st,
                      split > 1 ? static_cast<unsigned>(split) : 0u, a, units, static_cast<int>(split));
}

template <int TOK, int R>
lowbit_status launch_g(const GsArgs &a, cudaStream_t st)
{
    if (a.gshift == 8) return launch<TOK, kG256, R>(a, st);
    if (a.gshift == 7) return launch<TOK, kG128, R>(a, st);
    return a.gshift == 6 ? launch<TOK, kG64, R>(a, st) : launch<TOK, kG32, R>(a, st);
}

}  // namespace gsm

lowbit_status gs_mma_launch(const GsArgs &a, cudaStream_t st)
{
    const int64_t per = a.offsets != nullptr ? (a.M + a.E - 1) / a.E : a.M;
    if (per <= 8) return gsm::launch_g<8, 1>(a, st);
    if (per <= 16) return gsm::launch_g<16, 1>(a, st);
    return gsm::launch_g<32, 2>(a, st);
}

}  // namespace lowbit
