// gemv.hip -- products of a few tokens' bf16 activations with NVFP4 weights, for decoding:
//     y[t, j, n] = outer(r) sum_k x[t (, j), k] fp4(r, k) e4m3(r, k / 16),   r = ids[t, j] N + n
// per pair (t, j) of a token and its j-th expert, in fp32, bf16, or through SwiGLU (N = 2F).
//
// What bounds it: the weights' bytes from HBM, 9/16 of a byte each; next to them the vector instructions
// that unpack the codes (a CU has about 126 of them for 1 KB of codes at 5 TB/s).
//
// Split. A workgroup holds RT tiles of 16 rows of one expert's matrix (SwiGLU: 8 features of w1 and the same
// of w3) and all pairs that name the expert; its wavefronts share the contraction in units of 128 k, 64 bytes
// of codes of each row, dealt in turn: lane (g, i) loads the 16 bytes of row i that hold the unit's values
// 32 g .. 32 g + 31, one unit ahead of its use. The tiles' scales go through LDS in 16-byte pieces (loaded from
// memory per unit, 2 bytes a lane, they took a quarter of the time: one token through 8 experts of 4096 x 7168
// 37 us, 27 without any scales). The wavefronts' sums are added in order through LDS, so results do not
// depend on the launch.
//
// Up to two pairs (one decoded token): codes become bf16 exactly in one conversion for two, v_dot2_f32_bf16
// multiplies them with x from LDS, and a block's sum of 16 is multiplied by its scale once: 40 vector
// instructions for 32 weights and one pair. More pairs: fp4 * e4m3 has at most 6 significant bits and is exact
// in bf16 (two conversions and two products for two weights), for v_mfma_f32_16x16x32_bf16 with up to 16
// pairs as columns; more than 16 take the weights again, from the caches. Products are exact and sums fp32
// either way; the outer scales multiply the sums.
#include <type_traits>

#include "pmn_dev.hpp"
#include "pmn_kernels.hpp"

namespace pmn {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

struct GemvArgs {
    const uint16_t* x;        // [T x K], or [T*k x K] (per_pair)
    int per_pair;
    const uint8_t* codes;
    const uint8_t* scales;
    const float* outer;
    int64_t rpo;
    const int32_t* ids;       // [T*k], or null: matrix 0
    int k, G, pairs;
    int by_pair;              // workgroups go by pairs (the first of each expert works) or by experts
    int64_t N, K, F;
    int rblocks;              // workgroups a matrix
    void* out;                // [pairs x N], SwiGLU [pairs x F]
};

constexpr int GEMV_PAIRS = 4096;    // most pairs of a call
constexpr int GEMV_CHUNK = 8192;    // k whose scales (and x of two pairs) stand in LDS at a time
constexpr int GEMV_FEW = 2;         // pairs that go through dot2: a third and fourth in LDS would leave one workgroup a CU

static __device__ const uint4 gemv_zeros[4] = {};   // x past K: 32 values

PMN_DEV float dot2(uint32_t a, uint32_t b, float c)
{
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, a), __builtin_bit_cast(bf16x2, b), c, false);
}

// Byte `sel` of a code word, times a power of two, as two bf16
#define PMN_FP4_TO_BF16(w, two, sel) __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4((w), (two), (sel)))

// 8 codes times their scale d as bf16
PMN_DEV bf16x8 gemv_values(uint32_t codes, float d)
{
    float v[8];
    deq8(codes, d, v);
    const u32x4 b = {bf16x2_bits(v[0], v[1]), bf16x2_bits(v[2], v[3]), bf16x2_bits(v[4], v[5]), bf16x2_bits(v[6], v[7])};
    return __builtin_bit_cast(bf16x8, b);
}

// Outputs r0 .. of a pair that no expert computes (an id outside [0, G)): zeros.
PMN_DEV void gemv_zero(const GemvArgs& p, int pair, int64_t r0, int width, int64_t rows, int bytes)
{
    for (int i = threadIdx.x; i < width; i += blockDim.x)
        if (r0 + i < rows) {
            if (bytes == 4) static_cast<float*>(p.out)[(int64_t)pair * rows + r0 + i] = 0.0f;
            else static_cast<uint16_t*>(p.out)[(int64_t)pair * rows + r0 + i] = 0;
        }
}

template <int EPI, int RT, int W>
__global__ __launch_bounds__(W * 64, 4) void k_gemv(GemvArgs p, int pitch, int list0)
{
    constexpr bool SWI = EPI == PMN_EPI_SWIGLU;
    constexpr int RS = SWI ? 8 : 16, OB = EPI == PMN_EPI_F32 ? 4 : 2, THREADS = W * 64;
    // scales [RT * 16][pitch], then x of up to GEMV_FEW pairs in whole units; in their place at the end, the
    // wavefronts' sums red[W][RT][column][row]. From list0 the pairs of the expert.
    extern __shared__ __attribute__((aligned(16))) uint8_t dyn[];
    __shared__ int found[W];
    float (*red)[RT][16][16] = reinterpret_cast<float (*)[RT][16][16]>(dyn);
    uint16_t* const list = reinterpret_cast<uint16_t*>(dyn + list0);
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int l16 = lane & 15, g = lane >> 4;
    const int d = blockIdx.x / p.rblocks;
    const int64_t r0 = (int64_t)(blockIdx.x - d * p.rblocks) * (RT * RS);
    const int64_t rows = SWI ? p.F : p.N;
    const int K = (int)p.K;

    // this workgroup's expert, and the pairs that name it in their order
    int e = 0, n = p.pairs;
    if (p.ids && p.pairs <= 64) {
        const int id = lane < p.pairs ? p.ids[lane] : -1;
        e = p.by_pair ? __builtin_amdgcn_readlane(id, d) : d;
        if (e < 0 || e >= p.G) {   // by pairs only
            gemv_zero(p, d, r0, RT * RS, rows, OB);
            return;
        }
        if (!p.by_pair && d == 0) {
            uint64_t none = __ballot(lane < p.pairs && (id < 0 || id >= p.G));
            for (; none; none &= none - 1) gemv_zero(p, __builtin_ctzll(none), r0, RT * RS, rows, OB);
        }
        const uint64_t all = __ballot(id == e);
        if (all == 0 || (p.by_pair && __builtin_ctzll(all) != d)) return;   // an expert's first pair works for all
        n = __popcll(all);
        if (wave == 0 && id == e) list[__popcll(all & ((1ull << lane) - 1ull))] = (uint16_t)lane;
    } else if (p.ids) {
        e = p.by_pair ? __builtin_amdgcn_readfirstlane(p.ids[d]) : d;
        if (e < 0 || e >= p.G) {
            gemv_zero(p, d, r0, RT * RS, rows, OB);
            return;
        }
        n = 0;
        for (int base = 0; base < p.pairs; base += THREADS) {
            const int q = base + tid;
            const int id = q < p.pairs ? p.ids[q] : 0;
            const bool hit = q < p.pairs && id == e;
            const uint64_t all = __ballot(hit);
            if (lane == 0) found[wave] = __popcll(all);
            __syncthreads();
            int before = n;
#pragma unroll
            for (int v = 0; v < W; v++) {
                if (v < wave) before += found[v];
                n += found[v];
            }
            if (hit) list[before + __popcll(all & ((1ull << lane) - 1ull))] = (uint16_t)q;
            __syncthreads();
            if (!p.by_pair && d == 0 && __syncthreads_or(q < p.pairs && (id < 0 || id >= p.G))) {
                for (int b = base; b < base + THREADS && b < p.pairs; b++)
                    if (p.ids[b] < 0 || p.ids[b] >= p.G) gemv_zero(p, b, r0, RT * RS, rows, OB);
            }
        }
        if (n == 0 || (p.by_pair && list[0] != d)) return;
        n = __builtin_amdgcn_readfirstlane(n);
    }

    // rows of tile t, from the matrix' first (tiles past it repeat its first rows and are not stored)
    const uint8_t* base[RT];
#pragma unroll
    for (int t = 0; t < RT; t++)
        base[t] = p.codes + ((int64_t)e * p.N + (r0 + t * RS < rows ? r0 + t * RS : 0)) * (p.K >> 1);
    const uint32_t roff = (uint32_t)((SWI ? (l16 & 7) + (l16 >> 3) * p.F : l16) * (p.K >> 1));
    struct Batch {
        u32x4 c[RT];
    };
    auto load = [&](int u, Batch& b) {   // unit u; lanes past K read the row's last 32 again, times zeros
        int k = u * 128 + 32 * g;
        k = k < K ? k : K - 32;
#pragma unroll
        for (int t = 0; t < RT; t++) b.c[t] = *reinterpret_cast<const u32x4*>(base[t] + (roff + (uint32_t)(k >> 1)));
    };
    // the scales of k0 .. k0 + kn of all tiles' rows; rows begin at multiples of K / 16 bytes
    auto stage_scales = [&](int k0, int kn) {
        auto copy = [&](auto unit) {
            typedef decltype(unit) U;
            const int per = (kn >> 4) / (int)sizeof(U);
            for (int i = tid; i < RT * 16 * per; i += THREADS) {
                const int r = i / per, c = i - r * per, t = r >> 4;
                const int64_t first = r0 + t * RS < rows ? r0 + t * RS : 0;
                const int64_t row = (int64_t)e * p.N + first + (SWI ? (r & 7) + ((r >> 3) & 1) * p.F : r & 15);
                reinterpret_cast<U*>(dyn + r * pitch)[c] = reinterpret_cast<const U*>(p.scales + row * (p.K >> 4) + (k0 >> 4))[c];
            }
        };
        if (K % 256 == 0) copy(uint4{});
        else if (K % 64 == 0) copy(uint32_t{});
        else copy(uint16_t{});
    };
    // the two scales of this lane's 32 values of unit u (of its chunk) in tile t; not staged past K
    const uint8_t* const srow = dyn + l16 * pitch + 2 * g;
    auto scale_of = [&](int u, int t) -> uint32_t { return *reinterpret_cast<const uint16_t*>(srow + t * 16 * pitch + u * 8); };

    // sums of columns c0 .. c0 + nc - 1 from red
    auto finish = [&](int c0, int nc) {
        __syncthreads();
        for (int z = tid; z < RT * nc * (RS / 4); z += THREADS) {
            const int q = z % (RS / 4), c = z / (RS / 4) % nc, t = z / (RS / 4) / nc;
            const int64_t r = r0 + t * RS + 4 * q;
            if (r >= rows) continue;
            const int64_t pair = p.ids ? list[c0 + c] : c0 + c;
            float v[4] = {0.0f, 0.0f, 0.0f, 0.0f}, v3[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int w = 0; w < W; w++) {
                const float4 s = *reinterpret_cast<const float4*>(&red[w][t][c][4 * q]);
                v[0] += s.x; v[1] += s.y; v[2] += s.z; v[3] += s.w;
                if (SWI) {
                    const float4 s3 = *reinterpret_cast<const float4*>(&red[w][t][c][8 + 4 * q]);
                    v3[0] += s3.x; v3[1] += s3.y; v3[2] += s3.z; v3[3] += s3.w;
                }
            }
            const float o = p.outer[((int64_t)e * p.N + r) / p.rpo];
#pragma unroll
            for (int i = 0; i < 4; i++) v[i] *= o;
            if (SWI) {
                const float o3 = p.outer[((int64_t)e * p.N + p.F + r) / p.rpo];
#pragma unroll
                for (int i = 0; i < 4; i++) v[i] = silu(v[i]) * (v3[i] * o3);
            }
            if (EPI == PMN_EPI_F32) *reinterpret_cast<float4*>(static_cast<float*>(p.out) + pair * rows + r) = make_float4(v[0], v[1], v[2], v[3]);
            else *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + pair * rows + r) = make_uint2(bf16x2_bits(v[0], v[1]), bf16x2_bits(v[2], v[3]));
        }
    };

    // Chunks of the contraction with their scales in LDS (one for K up to GEMV_CHUNK), then this wavefront's
    // units of it with the next one's codes on their way. before(k0, kn) stages what else the chunk needs.
    auto contract = [&](auto before, auto compute) {
        for (int k0 = 0; k0 < K; k0 += GEMV_CHUNK) {
            const int kn = K - k0 < GEMV_CHUNK ? K - k0 : GEMV_CHUNK, u0 = k0 >> 7, un = (kn + 127) >> 7;
            Batch a, b;
            if (wave < un) load(u0 + wave, a);
            if (k0 > 0) __syncthreads();
            stage_scales(k0, kn);
            before(k0, kn);
            __syncthreads();
            for (int u = wave; u < un;) {
                if (u + W < un) load(u0 + u + W, b);
                compute(u0 + u, u, a);
                u += W;
                if (u >= un) break;
                if (u + W < un) load(u0 + u + W, a);
                compute(u0 + u, u, b);
                u += W;
            }
        }
    };

    if (n <= GEMV_FEW) {
        uint8_t* const xs = dyn + RT * 16 * pitch;
        constexpr int XROW = GEMV_CHUNK * 2;
        const int xrow = K < GEMV_CHUNK ? ((K + 127) >> 7) * 256 : XROW;
        auto run = [&](auto cols) {
            constexpr int C = decltype(cols)::value;
            float acc[C][RT];
#pragma unroll
            for (int c = 0; c < C; c++)
#pragma unroll
                for (int t = 0; t < RT; t++) acc[c][t] = 0.0f;
            contract(
                [&](int k0, int kn) {
                    if (k0 == 0 && p.ids && p.pairs <= 64) __syncthreads();   // list
#pragma unroll
                    for (int c = 0; c < C; c++) {
                        const int pair = p.ids ? list[c] : c;
                        const uint16_t* const x = p.x + (int64_t)(p.per_pair ? pair : pair / p.k) * p.K + k0;
                        for (int i = tid; i < ((kn + 127) >> 7) * 16; i += THREADS)
                            *reinterpret_cast<uint4*>(xs + c * xrow + i * 16) =
                                i * 8 < kn ? *reinterpret_cast<const uint4*>(x + i * 8) : make_uint4(0u, 0u, 0u, 0u);
                    }
                },
                [&](int uk, int u, const Batch& b) {
                    const bool in = uk * 128 + 32 * g < K;
                    uint32_t s[RT];
#pragma unroll
                    for (int t = 0; t < RT; t++) s[t] = in ? scale_of(u, t) : 0u;
#pragma unroll
                    for (int h = 0; h < 2; h++) {   // the lane's two blocks of 16
                        uint4 x[C][2];
#pragma unroll
                        for (int c = 0; c < C; c++)
#pragma unroll
                            for (int q = 0; q < 2; q++)
                                x[c][q] = *reinterpret_cast<const uint4*>(xs + c * xrow + u * 256 + g * 64 + h * 32 + q * 16);
#pragma unroll
                        for (int t = 0; t < RT; t++) {
                            // d16 = 2 two m: its power of two goes with the codes, so that the sum of 16 is no
                            // larger than the block's share of the result (with plain codes it passed fp32's range
                            // at |x| from 2^121 on), and 1/2 <= m < 1 with the sum, zero with a scale of zero
                            const float d16 = e4m3_value((s[t] >> (8 * h)) & 0xFFu);
                            const float two = __uint_as_float(__float_as_uint(d16) & 0x7F800000u);
                            const float m = __builtin_amdgcn_frexp_mantf(d16);
                            uint32_t v[8];
#pragma unroll
                            for (int q = 0; q < 2; q++) {
                                const uint32_t w = b.c[t][2 * h + q];
                                v[4 * q] = PMN_FP4_TO_BF16(w, two, 0);
                                v[4 * q + 1] = PMN_FP4_TO_BF16(w, two, 1);
                                v[4 * q + 2] = PMN_FP4_TO_BF16(w, two, 2);
                                v[4 * q + 3] = PMN_FP4_TO_BF16(w, two, 3);
                            }
#pragma unroll
                            for (int c = 0; c < C; c++) {
                                float sum = 0.0f;
#pragma unroll
                                for (int q = 0; q < 2; q++) {
                                    sum = dot2(v[4 * q], x[c][q].x, sum);
                                    sum = dot2(v[4 * q + 1], x[c][q].y, sum);
                                    sum = dot2(v[4 * q + 2], x[c][q].z, sum);
                                    sum = dot2(v[4 * q + 3], x[c][q].w, sum);
                                }
                                acc[c][t] = __builtin_fmaf(sum, m, acc[c][t]);
                            }
                        }
                    }
                });
#pragma unroll
            for (int c = 0; c < C; c++)
#pragma unroll
                for (int t = 0; t < RT; t++) {
                    float v = acc[c][t] * 2.0f;
                    v += __shfl_xor(v, 16, 64);
                    v += __shfl_xor(v, 32, 64);
                    acc[c][t] = v;
                }
            __syncthreads();
#pragma unroll
            for (int c = 0; c < C; c++)
#pragma unroll
                for (int t = 0; t < RT; t++)
                    if (g == 0) red[wave][t][c][l16] = acc[c][t];
        };
        if (n == 1) run(std::integral_constant<int, 1>{});
        else run(std::integral_constant<int, 2>{});
        finish(0, n);
        return;
    }

    if (p.ids && p.pairs <= 64) __syncthreads();   // list
    for (int c0 = 0; c0 < n; c0 += 16) {
        const int c = c0 + l16 < n ? c0 + l16 : n - 1;   // columns past the last repeat it
        const int pair = p.ids ? list[c] : c;
        const uint16_t* const xp = p.x + (int64_t)(p.per_pair ? pair : pair / p.k) * p.K;
        f32x4 acc[RT];
#pragma unroll
        for (int t = 0; t < RT; t++) acc[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        if (c0 > 0) __syncthreads();
        contract([](int, int) {},
                 [&](int uk, int u, const Batch& b) {
                     const int k = uk * 128 + 32 * g;
                     const bool in = k < K;
                     const uint16_t* const x = in ? xp + k : reinterpret_cast<const uint16_t*>(gemv_zeros);
                     bf16x8 f[4];
#pragma unroll
                     for (int s = 0; s < 4; s++) f[s] = *reinterpret_cast<const bf16x8*>(x + 8 * s);
#pragma unroll
                     for (int t = 0; t < RT; t++) {
                         const uint32_t sc = in ? scale_of(u, t) : 0u;
#pragma unroll
                         for (int s = 0; s < 4; s++)
                             acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                 gemv_values(b.c[t][s], e4m3_value((sc >> (8 * (s >> 1))) & 0xFFu)), f[s], acc[t], 0, 0, 0);
                     }
                 });
        __syncthreads();
#pragma unroll
        for (int t = 0; t < RT; t++)
            *reinterpret_cast<float4*>(&red[wave][t][l16][4 * g]) = make_float4(acc[t][0], acc[t][1], acc[t][2], acc[t][3]);
        finish(c0, n - c0 < 16 ? n - c0 : 16);
    }
}

int gemv_most_pairs() { return GEMV_PAIRS; }

// y of every pair: [T*k x N], SwiGLU [T*k x N/2]
hipError_t launch_gemv_pairs(const uint16_t* x, bool per_pair, const uint8_t* codes, const uint8_t* scales,
                             const float* outer, int64_t rpo, const int32_t* ids, int T, int k, int G, int64_t N,
                             int64_t K, int epilogue, void* out, hipStream_t stream)
{
    GemvArgs p{x, per_pair, codes, scales, outer, rpo, ids, k, G, T * k, 0, N, K, N / 2, 0, out};
    p.by_pair = ids && p.pairs < G;
    const int experts = !ids ? 1 : p.by_pair ? p.pairs : G;
    const int64_t tiles = epilogue == PMN_EPI_SWIGLU ? p.F / 8 : N / 16;
    // Wavefronts: a contraction of up to 4096 leaves 8 of them too few units each (5 tokens through 8 experts
    // of 7168 x 2048: 74 us with 8, 52 with 4; one of 4096 x 7168: 27 us with 8, 32 with 4). Tiles: three
    // where four rounds of workgroups are there (61 tokens, 4096 x 7168: 233 us with two, 212 with three: x is
    // read from L2 less often), two else (one token: 28 us with two, 30 with three), one where two would leave
    // CUs without a workgroup.
    const int w = K <= 4096 ? 4 : 8;
    auto groups = [&](int r) { return experts * ((tiles + r - 1) / r); };
    const int rt = groups(3) >= 4 * 256 * 16 / w ? 3 : groups(2) >= 512 ? 2 : 1;
    p.rblocks = (int)((tiles + rt - 1) / rt);
    const int chunk = K < GEMV_CHUNK ? (int)((K + 127) / 128 * 128) : GEMV_CHUNK;
    const int pitch = chunk / 16 + 16;   // 16 rows a dword apart hit different banks
    const int sums = w * rt * 1024, staged = rt * 16 * pitch + GEMV_FEW * chunk * 2, list0 = staged > sums ? staged : sums;
    const size_t lds = list0 + (p.pairs * 2 + 15) / 16 * 16;
    const dim3 grid((unsigned)(experts * p.rblocks)), block(w * 64);
    auto go = [&](auto epi, auto r, auto waves) {
        hipLaunchKernelGGL((k_gemv<decltype(epi)::value, decltype(r)::value, decltype(waves)::value>), grid, block, lds, stream, p, pitch, list0);
    };
    auto by_shape = [&](auto epi) {
        const std::integral_constant<int, 1> one;
        const std::integral_constant<int, 2> two;
        const std::integral_constant<int, 3> three;
        const std::integral_constant<int, 4> four;
        const std::integral_constant<int, 8> eight;
        if (w == 4) rt == 3 ? go(epi, three, four) : rt == 2 ? go(epi, two, four) : go(epi, one, four);
        else rt == 3 ? go(epi, three, eight) : rt == 2 ? go(epi, two, eight) : go(epi, one, eight);
    };
    if (epilogue == PMN_EPI_SWIGLU) by_shape(std::integral_constant<int, PMN_EPI_SWIGLU>{});
    else if (epilogue == PMN_EPI_F32) by_shape(std::integral_constant<int, PMN_EPI_F32>{});
    else by_shape(std::integral_constant<int, PMN_EPI_BF16>{});
    return hipGetLastError();
}

}  // namespace pmn
