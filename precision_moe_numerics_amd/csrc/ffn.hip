// ffn.hip -- the dense gated feed-forward block (the shared expert beside the routed ones) in bf16:
//     [h1 | h3] = x w13^T,  a = silu(h1) h3,  y = a w2^T (+ add)
// and its backward
//     da = dy w2,  dh1 = da h3 silu'(h1),  dh3 = da silu(h1)
//     dx = [dh1 | dh3] w13,  dw13 = [dh1 | dh3]^T x,  dw2 = dy^T a
// x, y, dy [M x H], w13 [2F x H] (w1 over w3), w2 [H x F], h13 [M x 2F], all row-major.
//
// Every product is out[c, r] = sum_k R(r, k) C(c, k) on v_mfma_f32_32x32x16_bf16 with fp32
// accumulators: "R" supplies the matrix rows (output features, so that a lane holds 4 consecutive
// ones of one output row), "C" the columns. An operand is either k-contiguous (rows of the matrix
// are rows of the product) or row-contiguous (the matrix is stored transposed: the weights in dgrad,
// both operands in wgrad).
#include "pmn_dev.hpp"
#include "pmn_kernels.hpp"

namespace pmn {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

namespace ffn {
constexpr int BT = 128, BK = 32, THREADS = 256, PITCH = BK + 8;
}

enum { FFN_SWIGLU = 0, FFN_ADD = 1, FFN_SWIGLU_BWD = 2, FFN_BF16 = 3, FFN_F32 = 4 };

struct FfnArgs {
    const uint16_t* r;      // R operand, ldr elements between its stored rows
    const uint16_t* c;
    int64_t ldr, ldc;
    int64_t Nr, Nc, K;      // product: Nc output rows x Nr output columns, contraction K
    void* out;              // [Nc x Nr] (SWIGLU: a [Nc x F]; SWIGLU_BWD: dh13 [Nc x 2F])
    const uint16_t* aux;    // ADD: add (or null); SWIGLU_BWD: h13
    uint16_t* out2;         // SWIGLU: h13 (or null); SWIGLU_BWD: a
    int64_t F;
};

// Stage a 128 x 32 operand tile as lds[row][k]. KC: 16-byte pieces of 8 k; else 8 rows at one k.
template <bool KC, typename RowOf>
PMN_DEV void stage_tile(const uint16_t* src, int64_t ld, int64_t nrows, int64_t k0, int64_t K, RowOf row_of,
                        uint16_t (*lds)[ffn::PITCH])
{
    using namespace ffn;
#pragma unroll
    for (int q = 0; q < BT * BK / 8 / THREADS; q++) {
        const int p = q * THREADS + threadIdx.x;
        uint4 w = make_uint4(0u, 0u, 0u, 0u);
        if (KC) {
            const int row = p >> 2, kc = (p & 3) * 8;
            const int64_t r = row_of(row);
            if (r >= 0 && k0 + kc < K) w = *reinterpret_cast<const uint4*>(src + r * ld + k0 + kc);
            *reinterpret_cast<uint4*>(&lds[row][kc]) = w;
        } else {
            const int k = p >> 4, rc = (p & 15) * 8;
            const int64_t r = row_of(rc);
            if (r >= 0 && k0 + k < K) w = *reinterpret_cast<const uint4*>(src + (k0 + k) * ld + r);
            const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int j = 0; j < 8; j++) lds[rc + j][k] = (uint16_t)(j & 1 ? a[j >> 1] >> 16 : a[j >> 1]);
        }
    }
}

template <bool RKC, bool CKC, int EPI>
__global__ __launch_bounds__(ffn::THREADS) void k_ffn_gemm(FfnArgs p)
{
    using namespace ffn;
    __shared__ __attribute__((aligned(16))) uint16_t lr[BT][PITCH], lc[BT][PITCH];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int wr = wave >> 1, wc = wave & 1, l32 = lane & 31, hh = lane >> 5;
    const int64_t c0 = (int64_t)blockIdx.y * BT;
    // SWIGLU: a tile holds 64 features, w1 and w3 rows of the same feature in blocks 0 and 1 of a wavefront
    const int64_t r0 = (int64_t)blockIdx.x * (EPI == FFN_SWIGLU ? BT / 2 : BT);
    auto row_r = [&](int t) -> int64_t {
        if (EPI == FFN_SWIGLU) {
            const int64_t f = r0 + (t >> 6) * 32 + (t & 31);
            return f < p.F ? ((t >> 5) & 1) * p.F + f : -1;
        }
        return r0 + t < p.Nr ? r0 + t : -1;
    };
    auto row_c = [&](int t) -> int64_t { return c0 + t < p.Nc ? c0 + t : -1; };
    f32x16 acc[2][2];
#pragma unroll
    for (int i = 0; i < 2; i++)
#pragma unroll
        for (int j = 0; j < 2; j++)
#pragma unroll
            for (int v = 0; v < 16; v++) acc[i][j][v] = 0.0f;
    for (int64_t k0 = 0; k0 < p.K; k0 += BK) {
        __syncthreads();
        stage_tile<RKC>(p.r, p.ldr, p.Nr, k0, p.K, row_r, lr);
        stage_tile<CKC>(p.c, p.ldc, p.Nc, k0, p.K, row_c, lc);
        __syncthreads();
#pragma unroll
        for (int ks = 0; ks < BK; ks += 16) {
            bf16x8 a[2], b[2];
#pragma unroll
            for (int i = 0; i < 2; i++) {
                a[i] = *reinterpret_cast<const bf16x8*>(&lr[wr * 64 + i * 32 + l32][ks + 8 * hh]);
                b[i] = *reinterpret_cast<const bf16x8*>(&lc[wc * 64 + i * 32 + l32][ks + 8 * hh]);
            }
#pragma unroll
            for (int i = 0; i < 2; i++)
#pragma unroll
                for (int j = 0; j < 2; j++)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[i], b[j], acc[i][j], 0, 0, 0);
        }
    }
#pragma unroll
    for (int j = 0; j < 2; j++) {
        const int64_t c = c0 + wc * 64 + j * 32 + l32;
        if (c >= p.Nc) continue;
#pragma unroll
        for (int i = 0; i < (EPI == FFN_SWIGLU ? 1 : 2); i++) {
#pragma unroll
            for (int q = 0; q < 4; q++) {
                const int64_t n = r0 + (EPI == FFN_SWIGLU ? wr * 32 : wr * 64 + i * 32) + q * 8 + hh * 4;
                if (n >= (EPI == FFN_SWIGLU ? p.F : p.Nr)) continue;   // sizes are multiples of 8
                float o[4];
#pragma unroll
                for (int u = 0; u < 4; u++) o[u] = acc[i][j][4 * q + u];
                auto put = [&](uint16_t* dst, const float (&v)[4]) {
                    *reinterpret_cast<uint2*>(dst) = make_uint2(bf16x2_bits(v[0], v[1]), bf16x2_bits(v[2], v[3]));
                };
                if (EPI == FFN_SWIGLU) {
                    float h3[4], a[4];
#pragma unroll
                    for (int u = 0; u < 4; u++) {
                        h3[u] = acc[1][j][4 * q + u];
                        a[u] = silu(o[u]) * h3[u];
                    }
                    put(static_cast<uint16_t*>(p.out) + c * p.F + n, a);
                    if (p.out2) {
                        put(p.out2 + c * 2 * p.F + n, o);
                        put(p.out2 + c * 2 * p.F + p.F + n, h3);
                    }
                } else if (EPI == FFN_SWIGLU_BWD) {
                    const uint2 w1 = *reinterpret_cast<const uint2*>(p.aux + c * 2 * p.F + n);
                    const uint2 w3 = *reinterpret_cast<const uint2*>(p.aux + c * 2 * p.F + p.F + n);
                    const float h1[4] = {bf16_lo(w1.x), bf16_hi(w1.x), bf16_lo(w1.y), bf16_hi(w1.y)};
                    const float h3[4] = {bf16_lo(w3.x), bf16_hi(w3.x), bf16_lo(w3.y), bf16_hi(w3.y)};
                    float d1[4], d3[4], a[4];
#pragma unroll
                    for (int u = 0; u < 4; u++) {
                        const float s = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-h1[u] * 1.44269504088896341f));
                        d1[u] = o[u] * h3[u] * (s * (1.0f + h1[u] * (1.0f - s)));
                        d3[u] = o[u] * h1[u] * s;
                        a[u] = h1[u] * s * h3[u];
                    }
                    put(static_cast<uint16_t*>(p.out) + c * 2 * p.F + n, d1);
                    put(static_cast<uint16_t*>(p.out) + c * 2 * p.F + p.F + n, d3);
                    put(p.out2 + c * p.F + n, a);
                } else if (EPI == FFN_F32) {
                    *reinterpret_cast<float4*>(static_cast<float*>(p.out) + c * p.Nr + n) =
                        make_float4(o[0], o[1], o[2], o[3]);
                } else {
                    if (EPI == FFN_ADD && p.aux) {
                        const uint2 w = *reinterpret_cast<const uint2*>(p.aux + c * p.Nr + n);
                        o[0] += bf16_lo(w.x); o[1] += bf16_hi(w.x); o[2] += bf16_lo(w.y); o[3] += bf16_hi(w.y);
                    }
                    put(static_cast<uint16_t*>(p.out) + c * p.Nr + n, o);
                }
            }
        }
    }
}

template <bool RKC, bool CKC, int EPI>
static void ffn_gemm(const FfnArgs& p, hipStream_t stream)
{
    const int64_t rt = ffn::BT / (EPI == FFN_SWIGLU ? 2 : 1), n = EPI == FFN_SWIGLU ? p.F : p.Nr;
    hipLaunchKernelGGL((k_ffn_gemm<RKC, CKC, EPI>), dim3((unsigned)((n + rt - 1) / rt), (unsigned)((p.Nc + ffn::BT - 1) / ffn::BT)),
                       dim3(ffn::THREADS), 0, stream, p);
}

// a [M x F] = silu(x w1^T) (x w3^T), with h13 where it is kept; y = a w2^T + add
hipError_t launch_ffn_fwd(const uint16_t* x, const uint16_t* w13, const uint16_t* w2, const uint16_t* add, int64_t M,
                          int64_t H, int64_t F, uint16_t* a, uint16_t* h13, uint16_t* y, hipStream_t stream)
{
    ffn_gemm<true, true, FFN_SWIGLU>(FfnArgs{w13, x, H, H, 2 * F, M, H, a, nullptr, h13, F}, stream);
    ffn_gemm<true, true, FFN_ADD>(FfnArgs{w2, a, F, F, H, M, F, y, add, nullptr, F}, stream);
    return hipGetLastError();
}

// dh13 [M x 2F] and a [M x F] from dy, w2 and h13; then the gradients asked for
hipError_t launch_ffn_bwd(const uint16_t* dy, const uint16_t* x, const uint16_t* w13, const uint16_t* w2,
                          const uint16_t* h13, int64_t M, int64_t H, int64_t F, uint16_t* dh13, uint16_t* a,
                          uint16_t* dx, void* dw13, void* dw2, bool dw_f32, hipStream_t stream)
{
    if (M > 0) ffn_gemm<false, true, FFN_SWIGLU_BWD>(FfnArgs{w2, dy, F, H, F, M, H, dh13, h13, a, F}, stream);
    if (M > 0 && dx) ffn_gemm<false, true, FFN_BF16>(FfnArgs{w13, dh13, H, 2 * F, H, M, 2 * F, dx, nullptr, nullptr, F}, stream);
    if (dw13) {
        const FfnArgs g13{x, dh13, H, 2 * F, H, 2 * F, M, dw13, nullptr, nullptr, F};
        const FfnArgs g2{a, dy, F, H, F, H, M, dw2, nullptr, nullptr, F};
        if (dw_f32) {
            ffn_gemm<false, false, FFN_F32>(g13, stream);
            ffn_gemm<false, false, FFN_F32>(g2, stream);
        } else {
            ffn_gemm<false, false, FFN_BF16>(g13, stream);
            ffn_gemm<false, false, FFN_BF16>(g2, stream);
        }
    }
    return hipGetLastError();
}

}  // namespace pmn
