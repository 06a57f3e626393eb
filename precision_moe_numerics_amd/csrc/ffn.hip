// ffn.hip -- the dense gated feed-forward block (the shared expert beside the routed ones) in bf16:
//     [h1 | h3] = x w13^T,  a = silu(h1) h3,  y = a w2^T (+ add)
// and its backward
//     da = dy w2,  dh1 = da h3 silu'(h1),  dh3 = da silu(h1)
//     dx = [dh1 | dh3] w13,  dw13 = [dh1 | dh3]^T x,  dw2 = dy^T a
// x, y, dy [M x H], w13 [2F x H] (w1 over w3), w2 [H x F], h13 [M x 2F], all row-major.
//
// Tiles, operand orders and the LDS ring: bf16_tile.hpp.
//
// a and dh13 are rounded to bf16 between the products, whose operands the bf16 MFMAs take (at most
// 2^-8 of a value; a second MFMA for what is rounded off would double those products): y and the gradients are
// off by 0.0021 to 0.0024 in norm, of which the rounding of the outputs themselves is 0.0017. h13 is stored
// in bf16; the forward's own a comes from the fp32 sums.
//
// Where the tiles of a product are fewer than the compute units the contraction is split: the parts
// write fp32 sums and a second kernel adds them in order and finishes the rows, so results do not
// depend on the launch.
#include "bf16_tile.hpp"
#include "pmn_kernels.hpp"

namespace pmn {

template <typename T, bool RKC, bool CKC, int EPI>
__global__ __launch_bounds__(T::THREADS, T::RB * T::CB == 16 ? 1 : 2) void k_ffn_gemm(FfnArgs p)
{
    __shared__ __attribute__((aligned(1024))) uint8_t lds[T::LDS];
    if (T::RB * T::CB == 16) asm volatile("; agpr in use %0" ::"a"(0));   // keeps the 256 accumulators in AGPRs
    int64_t L = blockIdx.x, trow, tcol;
    int split = 0;
    if (EPI == FFN_PART) {
        split = (int)(L % p.splits);
        L /= p.splits;
        trow = L % p.rtiles;
        tcol = L / p.rtiles;
    } else {
        if constexpr (T::HALVES) {
            // whole: all tiles, which need not fill the grid's last 8 workgroups, or a multiple of 256
            const int64_t rest = p.rtiles * p.ctiles - p.whole;
            if (rest > 0 && L >= p.whole) {
                const int64_t h = ffn_item_of(2 * rest, L - p.whole);
                if (h < 0) return;
                ffn_tile_at(p, p.whole + (h >> 1), trow, tcol);
                tcol = 2 * tcol + (h & 1);
                if (tcol * (T::BC / 2) < p.Nc) ffn_tile<typename T::Half, RKC, CKC, EPI>(p, trow, tcol, 0, lds);
                return;
            }
        }
        const int64_t i = ffn_item_of(T::HALVES ? p.whole : p.rtiles * p.ctiles, L);
        if (i < 0) return;
        ffn_tile_at(p, i, trow, tcol);
    }
    ffn_tile<T, RKC, CKC, EPI>(p, trow, tcol, split, lds);
}

// The gradients' products in one launch, weight gradients and dx in any order: workgroups up to end[0]
// work on p[0], up to end[1] on p[1], .. The chip stays full where one product's tiles run out, which
// with a launch each costs every product its last, partly filled round.
struct FfnGrads {
    FfnArgs p[3];
    uint32_t end[3];
    int dx;   // which of them is dx
};
template <typename T, int DW>
__global__ __launch_bounds__(T::THREADS, T::RB * T::CB == 16 ? 1 : 2) void k_ffn_grads(FfnGrads a)
{
    __shared__ __attribute__((aligned(1024))) uint8_t lds[T::LDS];
    if (T::RB * T::CB == 16) asm volatile("; agpr in use %0" ::"a"(0));
    const uint32_t L = blockIdx.x;
    const int w = L < a.end[0] ? 0 : L < a.end[1] ? 1 : 2;
    const uint32_t first = w == 0 ? 0u : w == 1 ? a.end[0] : a.end[1];
    const FfnArgs& p = a.p[w];
    int64_t trow, tcol;
    const int64_t i = ffn_item_of(p.rtiles * p.ctiles, L - first);
    if (i < 0) return;
    ffn_tile_at(p, i, trow, tcol);
    if (w == a.dx) ffn_tile<T, false, true, FFN_BF16>(p, trow, tcol, 0, lds);
    else ffn_tile<T, false, false, DW>(p, trow, tcol, 0, lds);
}

// Finish a split product: the parts of 8 consecutive outputs added in order. One thread each.
template <int EPI>
__global__ __launch_bounds__(256) void k_ffn_reduce(FfnArgs p)
{
    const int64_t per = (EPI == FFN_SWIGLU ? p.F : p.Nr) / 8;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= p.Nc * per) return;
    const int64_t c = i / per, n = (i - c * per) * 8;
    float v[8], v2[8];
    uint4 aux[2];
    ffn_aux8<EPI>(p, c, n, aux);
    auto sum = [&](int64_t col, float (&o)[8]) {
#pragma unroll
        for (int u = 0; u < 8; u++) o[u] = 0.0f;
#pragma unroll 4
        for (int s = 0; s < p.splits; s++) {
            const float4* src = reinterpret_cast<const float4*>(p.part + ((int64_t)s * p.Nc + c) * p.Nr + col);
            const float4 a = src[0], b = src[1];
            o[0] += a.x; o[1] += a.y; o[2] += a.z; o[3] += a.w;
            o[4] += b.x; o[5] += b.y; o[6] += b.z; o[7] += b.w;
        }
    };
    sum(n, v);
    if (EPI == FFN_SWIGLU) sum(p.F + n, v2);
    ffn_finish8<EPI>(p, c, n, v, v2, aux);
}

// A product for up to 16 output rows, both operands k-contiguous: the R operand, the weights, streams
// once from HBM and bounds it. A workgroup holds 16 rows of R (SWIGLU: 8 features of w1 and the same of
// w3) and its 8 wavefronts share the contraction in units of 64 k, one 128-byte line of each row, dealt
// in turn so that together they walk the rows; operands go straight to registers of
// v_mfma_f32_16x16x32_bf16, 4 units of a wavefront ahead, and the wavefronts' sums are added in order
// through LDS: one launch, no workspace. Columns past Nc repeat the last row and are not stored. Each
// workgroup reads all of C from L2, so beyond 16 rows the ring's tiles with a split contraction are
// faster (32 rows of 7168 x 2048: 35 us, this kernel with two column tiles 42).
// One row of 7168 x 2048 (88 MB of weights): 12.9 us and 7.8 us, 4.5 and 3.8 TB/s.
template <int EPI>
__global__ __launch_bounds__(512, 2) void k_ffn_few(FfnArgs p)
{
    constexpr bool SWI = EPI == FFN_SWIGLU;
    constexpr int W = 8, U = 4;
    __shared__ float4 red[W][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int l16 = lane & 15, g = lane >> 4;
    const int64_t r0 = (int64_t)blockIdx.x * (SWI ? 8 : 16);
    int64_t row = SWI ? r0 + (l16 & 7) : r0 + l16;
    const int64_t rows = SWI ? p.F : p.Nr;
    row = row < rows ? row : rows - 1;
    if (SWI && l16 >= 8) row += p.F;
    const uint16_t* const rp = p.r + row * p.ldr + 8 * g;
    const uint16_t* const cp = p.c + (l16 < p.Nc ? l16 : p.Nc - 1) * p.ldc + 8 * g;
    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
    const int64_t units = p.K >> 6;
    auto load = [](const uint16_t* q) { return *reinterpret_cast<const bf16x8*>(q); };
    // U units from unit u on; checked: chunks past K are zeros
    auto batch = [&](int64_t u, auto checked) {
        bf16x8 a[U][2], b[U][2];
#pragma unroll
        for (int i = 0; i < U; i++)
#pragma unroll
            for (int h = 0; h < 2; h++) {
                const int64_t k = (u + W * i) * 64 + 32 * h;
                if (!decltype(checked)::value || k + 8 * g < p.K) {
                    a[i][h] = load(rp + k);
                    b[i][h] = load(cp + k);
                } else {
                    a[i][h] = bf16x8{};
                    b[i][h] = bf16x8{};
                }
            }
#pragma unroll
        for (int i = 0; i < U; i++)
#pragma unroll
            for (int h = 0; h < 2; h++)
                acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[i][h], b[i][h], acc, 0, 0, 0);
    };
    int64_t u = wave;
    for (; u + W * (U - 1) < units; u += W * U) batch(u, std::false_type{});
    for (; u * 64 < p.K; u += W * U) batch(u, std::true_type{});
    red[wave][lane] = make_float4(acc[0], acc[1], acc[2], acc[3]);
    __syncthreads();
    if (wave > 0) return;
    // lane l finishes rows 4 (l / 16) .. +3 of column l % 16
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int w = 0; w < W; w++) {
        const float4 s = red[w][lane];
        v[0] += s.x; v[1] += s.y; v[2] += s.z; v[3] += s.w;
    }
    const int64_t c = l16;
    auto put = [](uint16_t* dst, const float (&o)[4]) {
        *reinterpret_cast<uint2*>(dst) = make_uint2(bf16x2_bits(o[0], o[1]), bf16x2_bits(o[2], o[3]));
    };
    if (SWI) {
        // lanes 0 .. 31 hold h1 of 8 features, lanes 32 .. 63 their h3
        float h3[4], a[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            h3[i] = __shfl_xor(v[i], 32, 64);
            a[i] = silu(v[i]) * h3[i];
        }
        const int64_t f = r0 + 4 * g;
        if (g >= 2 || c >= p.Nc || f >= p.F) return;
        put(static_cast<uint16_t*>(p.out) + c * p.F + f, a);
        if (p.out2) {
            put(p.out2 + c * 2 * p.F + f, v);
            put(p.out2 + c * 2 * p.F + p.F + f, h3);
        }
    } else {
        const int64_t n = r0 + 4 * g;
        if (c >= p.Nc || n >= p.Nr) return;
        if (p.aux) {
            const uint2 w = *reinterpret_cast<const uint2*>(p.aux + c * p.Nr + n);
            v[0] += bf16_lo(w.x); v[1] += bf16_hi(w.x); v[2] += bf16_lo(w.y); v[3] += bf16_hi(w.y);
        }
        put(static_cast<uint16_t*>(p.out) + c * p.Nr + n, v);
    }
}

typedef FfnTile<2, 2, 4, 4, 4> FfnLarge;    // 256 x 256, one workgroup per CU
typedef FfnTile<2, 2, 2, 2, 4> FfnMid;      // 128 x 128
typedef FfnTile<4, 1, 1, 2, 4> FfnFew;      // 128 x 64: few output rows, the R operand streams
typedef FfnTile<4, 1, 1, 2, 4, false> FfnShort;   // the same by single stages

constexpr int FFN_CUS = 256;   // the split's target; fixed, so that results depend on the sizes alone

struct FfnPlan {
    int tile;      // 0 large, 1 mid, 2 few
    int splits;    // 0: no split
};

// Tile and split of a product of Nc x Nr outputs over K. The small tiles split the contraction so that
// one workgroup, and no second one, goes to each CU: parts that leave a few CUs with two cost the length
// of one more (rounded up, not down: 384 rows of 7168 x 2048 forward 77 us against 61, 640 rows of 1024 x
// 2048 40 against 28). Large tiles from half a round of them: 128 x 128 ones would take 3000 rows of 4096 x
// 1536 140 us against 124; below that they are faster. 128 x 64 tiles, whose fewer parts are shorter to
// add but which load 1.5 times the bytes, where they are split in two or more, or three for a long
// contraction: 200 rows of 4096 x 1536 39 us against 34; with two parts of 7168, 160 rows of 7168 x 2048
// 43 us against 47. (Rounding down leaves CUs idle where a product has 129 to 255 tiles: 768 rows of 7168 x
// 2048 take 102 us where rounding up took 97, 1024 rows 112 against 110.)
static FfnPlan ffn_plan(int64_t Nc, int64_t Nr, int64_t K, bool ckc)
{
    if (Nc == 0) return {1, 0};
    auto tiles = [&](int64_t br, int64_t bc) { return ((Nr + br - 1) / br) * ((Nc + bc - 1) / bc); };
    const int64_t stages = (K + 31) / 32;
    auto split_for = [&](int64_t t, int64_t least) {
        int64_t s = FFN_CUS / t;
        const int64_t most = stages / least;
        s = s > most ? most : s;
        return (int)(s < 1 ? 1 : (s > 64 ? 64 : s));
    };
    const int64_t few = tiles(128, 64);
    if (ckc && (Nc <= 64 || (stages >= 32 && few <= (stages <= 128 ? FFN_CUS / 2 : FFN_CUS / 3))))
        return {2, split_for(few, 8)};
    if (tiles(256, 256) >= FFN_CUS / 2) return {0, 0};
    const int64_t t = tiles(128, 128);
    if (t >= FFN_CUS || stages < 32) return {1, 0};
    const int s = split_for(t, 16);
    return {1, s > 1 ? s : 0};
}

// Whether the 128 x 64 tiles load their part of the contraction by pairs of stages: where it is long enough for
// the pairs' prologue of five stages and, with k-contiguous weights, all parts begin on a whole line. (One product,
// contraction x columns, us by pairs / single stages: 17 tokens, 4096 x 2048 in parts of 8 stages, 6.7 / 6.5; 128 tokens,
// 7168 x 4096 in parts of 56, 18.7 / 21.9; 300 tokens, 7168 x 2048 in parts of 74 and 75, 21.5 / 19.4. Parts of 10 to
// 14 stages between 4% faster and 9% slower by pairs. Row-contiguous weights in parts of 74 and 75, the whole data
// gradient of 300 tokens through a block of 7168 x 2048: 60.6 / 61.4.)
static bool ffn_by_pairs(int64_t K, int splits, bool rkc)
{
    const int64_t stages = (K + 31) / 32;
    return stages >= 16 * splits && (!rkc || splits == 1 || stages % (2 * splits) == 0);
}

static int64_t ffn_part_floats(int64_t Nc, int64_t Nr, int64_t K, bool ckc)
{
    return (int64_t)ffn_plan(Nc, Nr, K, ckc).splits * Nc * Nr;
}

// Tile grid of a product; returns its workgroups (a multiple of 8, without PART). Where 256 x 256 tiles
// leave a last round with up to half of the CUs at work, that round's tiles go in halves to all of them
// (8192 x 7168 x 2048 forward, whose w2 product has 896: 621 -> 607 us); a fuller round would not fit in
// halves.
// halves: false in the gradients' launch, whose products fill each other's rounds.
template <typename T, int EPI>
static int64_t ffn_grid(FfnArgs& p, bool halves)
{
    const int64_t nr = EPI == FFN_SWIGLU ? p.F : p.Nr, br = EPI == FFN_SWIGLU ? T::BR / 2 : T::BR;
    p.rtiles = (nr + br - 1) / br;
    p.ctiles = (p.Nc + T::BC - 1) / T::BC;
    const int64_t n = p.rtiles * p.ctiles;
    if (EPI == FFN_PART) return n * p.splits;
    const int64_t rest = n % FFN_CUS;
    p.whole = T::HALVES && halves && rest > 0 && rest <= FFN_CUS / 2 ? n - rest : n;
    return p.whole < n ? p.whole + (2 * rest + 7) / 8 * 8 : (n + 7) / 8 * 8;
}

template <typename T, bool RKC, bool CKC, int EPI>
static void ffn_launch_tile(FfnArgs p, hipStream_t stream)
{
    const int64_t grid = ffn_grid<T, EPI>(p, true);
    hipLaunchKernelGGL((k_ffn_gemm<T, RKC, CKC, EPI>), dim3((unsigned)grid), dim3(T::THREADS), 0, stream, p);
}

// The gradients' products (count of them, dx at index dx or -1) in one launch, the longest contraction
// first
template <typename T, int DW>
static void ffn_launch_grads(const FfnArgs* p, int count, int dx, hipStream_t stream)
{
    int order[3] = {0, 1, 2};
    for (int i = 0; i < count; i++)
        for (int j = i + 1; j < count; j++)
            if (p[order[j]].K > p[order[i]].K) { const int t = order[i]; order[i] = order[j]; order[j] = t; }
    FfnGrads a{};
    a.dx = -1;
    int64_t end = 0;
    for (int i = 0; i < 3; i++) {
        if (i < count) {
            a.p[i] = p[order[i]];
            if (order[i] == dx) a.dx = i;
            end += ffn_grid<T, FFN_BF16>(a.p[i], false);
        }
        a.end[i] = (uint32_t)end;
    }
    hipLaunchKernelGGL((k_ffn_grads<T, DW>), dim3((unsigned)end), dim3(T::THREADS), 0, stream, a);
}

template <bool RKC, bool CKC, int EPI>
static void ffn_gemm(FfnArgs p, float* part, hipStream_t stream)
{
    if constexpr (RKC && CKC) {
        if (p.Nc <= 16) {
            const unsigned grid = (unsigned)(EPI == FFN_SWIGLU ? (p.F + 7) / 8 : (p.Nr + 15) / 16);
            hipLaunchKernelGGL((k_ffn_few<EPI>), dim3(grid), dim3(512), 0, stream, p);
            return;
        }
    }
    const FfnPlan pl = ffn_plan(p.Nc, p.Nr, p.K, CKC);
    p.splits = pl.splits;
    p.part = part;
    if (pl.splits == 0) {
        if (pl.tile == 0) ffn_launch_tile<FfnLarge, RKC, CKC, EPI>(p, stream);
        else ffn_launch_tile<FfnMid, RKC, CKC, EPI>(p, stream);
        return;
    }
    if (pl.tile == 1) ffn_launch_tile<FfnMid, RKC, CKC, FFN_PART>(p, stream);
    else if constexpr (CKC) {
        if (ffn_by_pairs(p.K, pl.splits, RKC)) ffn_launch_tile<FfnFew, RKC, CKC, FFN_PART>(p, stream);
        else ffn_launch_tile<FfnShort, RKC, CKC, FFN_PART>(p, stream);
    }
    const int64_t n = p.Nc * ((EPI == FFN_SWIGLU ? p.F : p.Nr) / 8);
    hipLaunchKernelGGL((k_ffn_reduce<EPI>), dim3((unsigned)((n + 255) / 256)), dim3(256), 0, stream, p);
}

size_t ffn_part_bytes(int64_t M, int64_t H, int64_t F, bool bwd)
{
    int64_t n = 0;
    auto need = [&](int64_t nc, int64_t nr, int64_t k, bool ckc) {
        const int64_t f = ffn_part_floats(nc, nr, k, ckc);
        n = f > n ? f : n;
    };
    if (!bwd) {
        need(M, 2 * F, H, true);
        need(M, H, F, true);
    } else {
        need(M, F, H, true);
        need(M, H, 2 * F, true);
        need(2 * F, H, M, false);
        need(H, F, M, false);
    }
    return (size_t)n * sizeof(float);
}

// a [M x F] = silu(x w1^T) (x w3^T), with h13 where it is kept; y = a w2^T + add
hipError_t launch_ffn_fwd(const uint16_t* x, const uint16_t* w13, const uint16_t* w2, const uint16_t* add, int64_t M,
                          int64_t H, int64_t F, uint16_t* a, float* part, uint16_t* h13, uint16_t* y, hipStream_t stream)
{
    ffn_gemm<true, true, FFN_SWIGLU>(FfnArgs{w13, x, H, H, 2 * F, M, H, a, nullptr, h13, F}, part, stream);
    ffn_gemm<true, true, FFN_ADD>(FfnArgs{w2, a, F, F, H, M, F, y, add, nullptr, F}, part, stream);
    return hipGetLastError();
}

// Tile of the gradients' one launch, -1 for a launch each with split contractions. One launch where
// its workgroups fill the chip and the longest contraction is not much longer than their share of it:
// with few tiles of a long one (small weights, many tokens) splitting them is faster. 256 x 256 tiles from
// 640 of them, two and a half rounds: 7 to 17% faster than 128 x 128 ones at 640 to 944 (4096 rows of 4096 x
// 2048: 377 us against 411). Below, from 416 on, between 3% slower (2000 rows of 7168 x 1024, 560 tiles: 209
// us against 203) and 13% faster (3100 of 4096 x 1536, 496: 233 against 267), at 304 to 320 7 to 11% slower.
static int ffn_grads_tile(int64_t M, int64_t H, int64_t F, bool dgrad, bool wgrad)
{
    if (M == 0) return 1;
    int64_t tiles[2] = {0, 0}, steps[2] = {0, 0}, longest = 0;
    auto count = [&](int64_t nc, int64_t nr, int64_t k) {
        const int64_t st = (k + 31) / 32;
        longest = st > longest ? st : longest;
        for (int i = 0; i < 2; i++) {
            const int64_t b = i == 0 ? 256 : 128, t = ((nr + b - 1) / b) * ((nc + b - 1) / b);
            tiles[i] += t;
            steps[i] += t * st;
        }
    };
    if (wgrad) {
        count(2 * F, H, M);
        count(H, F, M);
    }
    if (dgrad) count(M, H, 2 * F);
    if (tiles[0] >= 640 && longest * FFN_CUS <= steps[0]) return 0;
    if (tiles[1] >= FFN_CUS && longest * FFN_CUS <= steps[1]) return 1;
    return -1;
}

// dh13 [M x 2F] and a [M x F] from dy, w2 and h13; then the gradients asked for
hipError_t launch_ffn_bwd(const uint16_t* dy, const uint16_t* x, const uint16_t* w13, const uint16_t* w2,
                          const uint16_t* h13, int64_t M, int64_t H, int64_t F, uint16_t* dh13, uint16_t* a,
                          float* part, uint16_t* dx, void* dw13, void* dw2, bool dw_f32, hipStream_t stream)
{
    if (M > 0) ffn_gemm<false, true, FFN_SWIGLU_BWD>(FfnArgs{w2, dy, F, H, F, M, H, dh13, h13, a, F}, part, stream);
    FfnArgs g[3];
    int count = 0, idx = -1;
    if (dw13) {
        g[count++] = FfnArgs{x, dh13, H, 2 * F, H, 2 * F, M, dw13, nullptr, nullptr, F};
        g[count++] = FfnArgs{a, dy, F, H, F, H, M, dw2, nullptr, nullptr, F};
    }
    if (M > 0 && dx) {
        idx = count;
        g[count++] = FfnArgs{w13, dh13, H, 2 * F, H, M, 2 * F, dx, nullptr, nullptr, F};
    }
    const int tile = ffn_grads_tile(M, H, F, dx != nullptr, dw13 != nullptr);
    if (tile >= 0) {
        if (tile == 0) {
            if (dw_f32) ffn_launch_grads<FfnLarge, FFN_F32>(g, count, idx, stream);
            else ffn_launch_grads<FfnLarge, FFN_BF16>(g, count, idx, stream);
        } else {
            if (dw_f32) ffn_launch_grads<FfnMid, FFN_F32>(g, count, idx, stream);
            else ffn_launch_grads<FfnMid, FFN_BF16>(g, count, idx, stream);
        }
        return hipGetLastError();
    }
    for (int i = 0; i < count; i++) {
        if (i == idx) ffn_gemm<false, true, FFN_BF16>(g[i], part, stream);
        else if (dw_f32) ffn_gemm<false, false, FFN_F32>(g[i], part, stream);
        else ffn_gemm<false, false, FFN_BF16>(g[i], part, stream);
    }
    return hipGetLastError();
}

}  // namespace pmn
