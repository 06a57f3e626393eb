// gemv.hip -- products of a few tokens' bf16 activations with NVFP4 weights, for decoding:
//     y[t, j, n] = outer(r) sum_k x[t (, j), k] fp4(r, k) e4m3(r, k / 16),   r = ids[t, j] N + n
// per pair (t, j) of a token and its j-th expert (k_gemv_pairs: fp32, bf16, or SwiGLU with N = 2F), or
// summed over a token's experts with its gates (k_gemv_sum).
//
// Arithmetic. fp4 * e4m3 has at most 6 significant bits and is exact in bf16, so the weights go to
// v_mfma_f32_16x16x32_bf16 as bf16 (one conversion to two fp32, two products by the block's scale, one
// packed conversion for two weights) and every product is exact; sums are fp32, outer scales and gates
// multiply the sums.
//
// What bounds it: the weights' bytes from HBM, 9/16 of a byte each. A workgroup holds 16 rows of a matrix
// (SwiGLU: 8 features of w1 and the same of w3) and its 8 wavefronts share the contraction in units of
// 128 k, 64 bytes of codes of each row: lane (g, i) loads 16 bytes of row i, the 32 values 32 g .. of the
// unit, with their two scale bytes; its 8 values of MFMA step s are 32 g + 8 s .., for both operands, so
// nothing is exchanged between lanes. Activations come from L2 straight to registers. The wavefronts' sums
// are added in order through LDS: results do not depend on the launch, and a column's not on the others.
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
    const float* gates;       // k_gemv_sum
    const uint16_t* add;      // k_gemv_sum: bf16 [T x N] or null
    int T, k, G, pairs;       // pairs = T * k
    int by_pair;              // workgroups go by pairs (the first of each expert works) or by experts
    int64_t N, K, F;
    int rblocks;
    void* out;
};

constexpr int GEMV_PAIRS = 4096;   // most pairs of a call
constexpr int GEMV_W = 8;          // wavefronts of a workgroup

// One unit of a lane: its codes and scales
struct GemvWeights {
    u32x4 c;
    uint32_t s;
};
PMN_DEV GemvWeights gemv_load(const uint8_t* codes, const uint8_t* scales, int64_t k, int64_t K)
{
    GemvWeights w{};
    if (k < K) {   // K % 32 == 0: a lane's 32 values are all inside or all outside
        w.c = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(codes + (k >> 1)));
        w.s = *reinterpret_cast<const uint16_t*>(scales + (k >> 4));
    }
    return w;
}

// The 8 weights of step s as bf16
PMN_DEV bf16x8 gemv_values(const GemvWeights& w, int s)
{
    const float d = e4m3_value((w.s >> (8 * (s >> 1))) & 0xFFu);
    float v[8];
    deq8(w.c[s], d, v);
    const u32x4 b = {bf16x2_bits(v[0], v[1]), bf16x2_bits(v[2], v[3]), bf16x2_bits(v[4], v[5]), bf16x2_bits(v[6], v[7])};
    return __builtin_bit_cast(bf16x8, b);
}

PMN_DEV bf16x8 gemv_x(const uint16_t* x, int64_t k, int64_t K)
{
    return k < K ? *reinterpret_cast<const bf16x8*>(x + k) : bf16x8{};
}

// Rows of a pair's outputs that nothing computes (an id outside [0, G)): zeros.
PMN_DEV void gemv_zero(const GemvArgs& p, int pair, int64_t r0, int width, int64_t rows, int bytes)
{
    for (int i = threadIdx.x; i < width; i += blockDim.x)
        if (r0 + i < rows) {
            if (bytes == 4) static_cast<float*>(p.out)[(int64_t)pair * rows + r0 + i] = 0.0f;
            else static_cast<uint16_t*>(p.out)[(int64_t)pair * rows + r0 + i] = 0;
        }
}

// A workgroup: 16 rows of one expert's matrix times the rows of all pairs that name it, in passes of
// 16 CT columns.
template <int EPI, int CT>
__global__ __launch_bounds__(GEMV_W * 64, 2) void k_gemv_pairs(GemvArgs p)
{
    constexpr bool SWI = EPI == PMN_EPI_SWIGLU;
    constexpr int W = GEMV_W, U = CT == 1 ? 4 : 2;
    __shared__ float4 red[W][CT][64];
    __shared__ uint16_t list[GEMV_PAIRS];
    __shared__ int found[W];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int l16 = lane & 15, g = lane >> 4;
    const int d = blockIdx.x / p.rblocks;
    const int64_t r0 = (int64_t)(blockIdx.x - d * p.rblocks) * (SWI ? 8 : 16);
    const int64_t rows = SWI ? p.F : p.N;
    constexpr int OB = EPI == PMN_EPI_F32 ? 4 : 2;
    const int e = !p.ids ? 0 : p.by_pair ? __builtin_amdgcn_readfirstlane(p.ids[d]) : d;
    if (e < 0 || e >= p.G) {   // by pairs only
        gemv_zero(p, d, r0, SWI ? 8 : 16, rows, OB);
        return;
    }
    int64_t row = SWI ? r0 + (l16 & 7) : r0 + l16;
    if (SWI && l16 >= 8) row += p.F;
    const int64_t at = (int64_t)e * p.N + row;
    const uint8_t* const codes = p.codes + at * (p.K >> 1);
    const uint8_t* const scales = p.scales + at * (p.K >> 4);
    const int64_t units = (p.K + 127) >> 7;

    // the pairs of this expert are listed in their order; a dense product's first weights are on their way
    // by then (an expert that no pair names reads nothing)
    GemvWeights w[U];
    auto load_weights = [&](int64_t u) {
#pragma unroll
        for (int i = 0; i < U; i++) w[i] = gemv_load(codes, scales, (u + W * i) * 128 + 32 * g, p.K);
    };
    if (!p.ids) load_weights(wave);
    int n = 0;
    for (int base = 0; base < p.pairs; base += W * 64) {
        const int q = base + tid;
        const int id = q < p.pairs ? (p.ids ? p.ids[q] : 0) : -1;
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
            for (int b = base; b < base + W * 64 && b < p.pairs; b++)
                if (p.ids[b] < 0 || p.ids[b] >= p.G) gemv_zero(p, b, r0, SWI ? 8 : 16, rows, OB);
        }
    }
    if (n == 0 || (p.by_pair && list[0] != d)) return;   // an expert's first pair works for all
    if (p.ids) load_weights(wave);

    for (int c0 = 0; c0 < n; c0 += 16 * CT) {
        const uint16_t* xp[CT];
        bool in[CT];
#pragma unroll
        for (int t = 0; t < CT; t++) {
            in[t] = c0 + 16 * t < n;   // uniform
            const int c = c0 + 16 * t + l16 < n ? c0 + 16 * t + l16 : n - 1;   // columns past the last repeat it
            const int pair = list[c];
            xp[t] = p.x + (int64_t)(p.per_pair ? pair : pair / p.k) * p.K;
        }
        f32x4 acc[CT];
#pragma unroll
        for (int t = 0; t < CT; t++) acc[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        if (c0 > 0) load_weights(wave);
        for (int64_t u = wave; u < units; u += W * U) {
            GemvWeights cur[U];
#pragma unroll
            for (int i = 0; i < U; i++) cur[i] = w[i];
            load_weights(u + W * U);
#pragma unroll
            for (int i = 0; i < U; i++) {
                const int64_t k = (u + W * i) * 128 + 32 * g;
                if ((u + W * i) >= units) break;
                bf16x8 x[CT][4];
#pragma unroll
                for (int t = 0; t < CT; t++)
                    if (in[t])
#pragma unroll
                        for (int s = 0; s < 4; s++) x[t][s] = gemv_x(xp[t], k < p.K ? k + 8 * s : p.K, p.K);
#pragma unroll
                for (int s = 0; s < 4; s++) {
                    const bf16x8 v = gemv_values(cur[i], s);
#pragma unroll
                    for (int t = 0; t < CT; t++)
                        if (in[t]) acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, x[t][s], acc[t], 0, 0, 0);
                }
            }
        }
        if (c0 > 0) __syncthreads();
#pragma unroll
        for (int t = 0; t < CT; t++)
            if (in[t]) red[wave][t][lane] = make_float4(acc[t][0], acc[t][1], acc[t][2], acc[t][3]);
        __syncthreads();
        // wavefront t finishes column tile t: lane l rows 4 (l / 16) .. +3 of column l % 16
        if (wave < CT && c0 + 16 * wave < n) {
            float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int q = 0; q < W; q++) {
                const float4 s = red[q][wave][lane];
                v[0] += s.x; v[1] += s.y; v[2] += s.z; v[3] += s.w;
            }
            const int c = c0 + 16 * wave + l16;
            // rows_per_outer is a multiple of 32: one scale for the rows of a workgroup's matrix
            const int64_t first = (int64_t)e * p.N + r0 + (SWI && g >= 2 ? p.F : 0);
            const float o = p.outer[first / p.rpo];
#pragma unroll
            for (int i = 0; i < 4; i++) v[i] *= o;
            if (SWI) {
                // lanes 0 .. 31 hold h1 of 8 features, lanes 32 .. 63 their h3
                float a[4];
#pragma unroll
                for (int i = 0; i < 4; i++) a[i] = silu(v[i]) * __shfl_xor(v[i], 32, 64);
                if (g < 2 && c < n)
                    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + (int64_t)list[c] * p.F + r0 + 4 * g) =
                        make_uint2(bf16x2_bits(a[0], a[1]), bf16x2_bits(a[2], a[3]));
            } else if (c < n) {
                const int64_t o4 = (int64_t)list[c] * p.N + r0 + 4 * g;
                if (EPI == PMN_EPI_F32) *reinterpret_cast<float4*>(static_cast<float*>(p.out) + o4) = make_float4(v[0], v[1], v[2], v[3]);
                else *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + o4) = make_uint2(bf16x2_bits(v[0], v[1]), bf16x2_bits(v[2], v[3]));
            }
        }
    }
}

// out[t, n] = sum_j gates[t, j] y[t, j, n] (+ add[t, n]) for up to 16 tokens: a workgroup holds 16 rows n of
// every expert that is named and adds its experts' sums, each with its tokens' gates, before the
// wavefronts' are joined. The work is a list of (expert, occurrence in its token): a token that names an
// expert twice has it in two entries. Its units go round the wavefronts, so one token's 8 experts of 2048
// k keep all of them at work.
template <bool F32OUT>
__global__ __launch_bounds__(GEMV_W * 64, 2) void k_gemv_sum(GemvArgs p)
{
    constexpr int W = GEMV_W, U = 4, MOST = 256;
    __shared__ float4 red[W][64];
    __shared__ int32_t id[MOST], key[MOST];
    __shared__ int16_t map[MOST][16];   // entry, token -> pair or -1
    __shared__ int32_t expert[MOST];
    __shared__ int found[W];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int l16 = lane & 15, g = lane >> 4;
    const int64_t r0 = (int64_t)blockIdx.x * 16;
    // pair q: its expert and which of its token's pairs with that expert it is
    int mine = -1;
    if (tid < p.pairs) {
        mine = p.ids ? p.ids[tid] : 0;
        if (mine < 0 || mine >= p.G) mine = -1;
        id[tid] = mine;
    }
    for (int i = tid; i < MOST * 16 / 2; i += W * 64) reinterpret_cast<uint32_t*>(map)[i] = 0xFFFFFFFFu;
    __syncthreads();
    int k = -1;
    if (mine >= 0) {
        int rank = 0;
        for (int q = tid / p.k * p.k; q < tid; q++) rank += id[q] == mine;
        k = mine * 16 + rank;   // at most 16 pairs a token
    }
    if (tid < p.pairs) key[tid] = k;
    __syncthreads();
    int first = tid;
    if (k >= 0)
        for (int q = 0; q < tid; q++)
            if (key[q] == k) {
                first = q;
                break;
            }
    const bool leads = k >= 0 && first == tid;
    const uint64_t all = __ballot(leads);
    if (lane == 0) found[wave] = __popcll(all);
    __syncthreads();
    int before = 0, entries = 0;
#pragma unroll
    for (int v = 0; v < W; v++) {
        if (v < wave) before += found[v];
        entries += found[v];
    }
    before += __popcll(all & ((1ull << lane) - 1ull));
    if (leads) {
        expert[before] = mine;
        id[tid] = before;   // the entry of the pairs that tid leads
    }
    __syncthreads();
    if (k >= 0) map[id[first]][tid / p.k] = (int16_t)tid;
    __syncthreads();

    const int units = (int)((p.K + 127) >> 7);
    const int items = entries * units;
    f32x4 total = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int it = wave; it < items; it += W * U) {
        GemvWeights w[U];
        bf16x8 x[U][4];
        float scale[U];
        bool on[U];   // the lane's token names the entry's expert: nothing is added otherwise, NaN scales neither
#pragma unroll
        for (int i = 0; i < U; i++) {
            const int item = it + W * i;
            w[i] = GemvWeights{};
            scale[i] = 0.0f;
            on[i] = false;
#pragma unroll
            for (int s = 0; s < 4; s++) x[i][s] = bf16x8{};
            if (item < items) {
                const int d = item / units;
                const int64_t kk = (int64_t)(item - d * units) * 128 + 32 * g;
                const int64_t at = (int64_t)__builtin_amdgcn_readfirstlane(expert[d]) * p.N + r0;
                w[i] = gemv_load(p.codes + (at + l16) * (p.K >> 1), p.scales + (at + l16) * (p.K >> 4), kk, p.K);
                const int pair = map[d][l16];
                if (pair >= 0) {
                    on[i] = true;
                    scale[i] = p.gates[pair] * p.outer[at / p.rpo];
                    const uint16_t* const xp = p.x + (int64_t)(p.per_pair ? pair : pair / p.k) * p.K;
#pragma unroll
                    for (int s = 0; s < 4; s++) x[i][s] = gemv_x(xp, kk < p.K ? kk + 8 * s : p.K, p.K);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < U; i++) {
            if (it + W * i >= items) break;
            f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int s = 0; s < 4; s++) acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(gemv_values(w[i], s), x[i][s], acc, 0, 0, 0);
#pragma unroll
            for (int q = 0; q < 4; q++) total[q] = on[i] ? __builtin_fmaf(acc[q], scale[i], total[q]) : total[q];
        }
    }
    red[wave][lane] = make_float4(total[0], total[1], total[2], total[3]);
    __syncthreads();
    if (wave > 0 || l16 >= p.T) return;
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int q = 0; q < W; q++) {
        const float4 s = red[q][lane];
        v[0] += s.x; v[1] += s.y; v[2] += s.z; v[3] += s.w;
    }
    const int64_t o = l16 * p.N + r0 + 4 * g;
    if (p.add) {
        const uint2 a = *reinterpret_cast<const uint2*>(p.add + o);
        v[0] += bf16_lo(a.x); v[1] += bf16_hi(a.x); v[2] += bf16_lo(a.y); v[3] += bf16_hi(a.y);
    }
    if (F32OUT) *reinterpret_cast<float4*>(static_cast<float*>(p.out) + o) = make_float4(v[0], v[1], v[2], v[3]);
    else *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + o) = make_uint2(bf16x2_bits(v[0], v[1]), bf16x2_bits(v[2], v[3]));
}

int gemv_most_pairs() { return GEMV_PAIRS; }
bool gemv_sums_at_once(int T, int k) { return T <= 16 && k <= 16; }

// y of every pair: [T*k x N], SwiGLU [T*k x N/2]
hipError_t launch_gemv_pairs(const uint16_t* x, bool per_pair, const uint8_t* codes, const uint8_t* scales,
                             const float* outer, int64_t rpo, const int32_t* ids, int T, int k, int G, int64_t N,
                             int64_t K, int epilogue, void* out, hipStream_t stream)
{
    GemvArgs p{x, per_pair, codes, scales, outer, rpo, ids, nullptr, nullptr, T, k, G, T * k, 0, N, K, N / 2, 0, out};
    p.by_pair = ids && p.pairs < G;
    p.rblocks = (int)(epilogue == PMN_EPI_SWIGLU ? p.F / 8 : N / 16);
    const int experts = !ids ? 1 : p.by_pair ? p.pairs : G;
    const dim3 grid((unsigned)(experts * p.rblocks)), block(GEMV_W * 64);
    // columns of an expert: one tile of 16 where no more tokens are there
    if (T <= 16) {
        if (epilogue == PMN_EPI_SWIGLU) hipLaunchKernelGGL((k_gemv_pairs<PMN_EPI_SWIGLU, 1>), grid, block, 0, stream, p);
        else if (epilogue == PMN_EPI_F32) hipLaunchKernelGGL((k_gemv_pairs<PMN_EPI_F32, 1>), grid, block, 0, stream, p);
        else hipLaunchKernelGGL((k_gemv_pairs<PMN_EPI_BF16, 1>), grid, block, 0, stream, p);
    } else {
        if (epilogue == PMN_EPI_SWIGLU) hipLaunchKernelGGL((k_gemv_pairs<PMN_EPI_SWIGLU, 4>), grid, block, 0, stream, p);
        else if (epilogue == PMN_EPI_F32) hipLaunchKernelGGL((k_gemv_pairs<PMN_EPI_F32, 4>), grid, block, 0, stream, p);
        else hipLaunchKernelGGL((k_gemv_pairs<PMN_EPI_BF16, 4>), grid, block, 0, stream, p);
    }
    return hipGetLastError();
}

// The gates' sum over up to 16 tokens and 16 experts each (gemv_sums_at_once)
hipError_t launch_gemv_sum(const uint16_t* x, bool per_pair, const uint8_t* codes, const uint8_t* scales,
                           const float* outer, int64_t rpo, const int32_t* ids, const float* gates,
                           const uint16_t* add, int T, int k, int G, int64_t N, int64_t K, bool f32, void* out,
                           hipStream_t stream)
{
    GemvArgs p{x, per_pair, codes, scales, outer, rpo, ids, gates, add, T, k, G, T * k, 0, N, K, 0, (int)(N / 16), out};
    const dim3 grid((unsigned)(N / 16)), block(GEMV_W * 64);
    if (f32) hipLaunchKernelGGL((k_gemv_sum<true>), grid, block, 0, stream, p);
    else hipLaunchKernelGGL((k_gemv_sum<false>), grid, block, 0, stream, p);
    return hipGetLastError();
}

}  // namespace pmn
