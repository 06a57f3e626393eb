// gemm_bf16.hip -- bf16 products grouped by expert, for layers (or passes) that are not quantized:
//     forward  Y[s, n] = sum_k x[row_s, k] W_g[n, k]        (bf16, fp32, or SwiGLU with h1 | h3 saved)
//     dgrad    da[s, k] = sum_n dY[s, n] W_g[n, k]          (or on through the SwiGLU: dh13)
//     wgrad    dW_g[n, k] = sum_{s in g} dY[s, n] x[row_s, k]
// g the group of slot s, row_s = gather[s] or s. Group sizes are on the device only.
//
// The tiles are bf16_tile.hpp's. Forward and dgrad run over the concatenation of the groups' units of
// BC slots; a workgroup finds its unit with one wavefront-parallel search of the offsets, and a unit of
// at most BC / 2 slots that ends a group runs as half a tile. Wgrad runs over the groups' (n, k) tiles,
// each of its group's length; a group without slots writes zeros.
//
// Sums are fp32; outputs are rounded once.
#include "bf16_tile.hpp"
#include "pmn_kernels.hpp"

namespace pmn {

struct GroupArgs {
    FfnArgs p;                // of the whole matrices; a workgroup moves the pointers to its group
    const int64_t* offsets;
    int G;
    int64_t rgroup;           // elements of R between groups' matrices
    int64_t out_width;        // output elements of a slot, and bytes of each
    int out_bytes;
    int64_t out2_width;
    bool apart;               // half tiles run after the whole ones
    int splits;               // parts of a group's slots in wgrad
};

// Moves p to group g, whose slots are s0 .. s1
template <bool GATHER>
PMN_DEV void group_at(const GroupArgs& a, int g, int64_t s0, int64_t s1, FfnArgs& p)
{
    p = a.p;
    p.r += g * a.rgroup;
    if (GATHER) p.gather += s0;
    else p.c += s0 * p.ldc;
    p.Nc = s1 - s0;
    p.out = static_cast<uint8_t*>(p.out) + s0 * a.out_width * a.out_bytes;
    if (p.out2) p.out2 += s0 * a.out2_width;
    if (p.aux) p.aux += s0 * 2 * p.F;
}

// Units over all groups, count(slots) each, on the device.
template <typename F>
PMN_DEV int64_t group_units(const int64_t* offsets, int G, F count)
{
    const int lane = threadIdx.x & 63;
    int64_t n = 0;
    for (int g = lane; g < G; g += 64) n += count(offsets[g + 1] - offsets[g]);
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) n += __shfl_xor(n, d, 64);
    return n;
}

PMN_DEV int64_t uniform64(int64_t v)
{
    const uint32_t lo = __builtin_amdgcn_readfirstlane((int)(uint32_t)v), hi = __builtin_amdgcn_readfirstlane((int)(uint32_t)(v >> 32));
    return (int64_t)((uint64_t)hi << 32 | lo);
}

// Item of workgroup L among n: each XCD takes 32 consecutive ones of every 256 (of what is left at the end, an
// eighth), so that all of them work on the same few groups at a time, whose operands the last-level cache holds:
// tiles of an XCD drift apart where some are halves, and miss its L2 (65536 slots in 48 groups of 4096 x 7168,
// each XCD on an eighth of all items 3326 us, so 3229; in blocks of 512 and 1024 1 and 2% slower). Negative past
// the last.
PMN_DEV int64_t group_item_of(int64_t n, int64_t L)
{
    const int64_t b = L >> 8, r = L & 255, left = n - (b << 8);
    const int64_t per = left < 256 ? (left + 7) >> 3 : 32, i = (r & 7) * per + (r >> 3);
    return (r >> 3) >= per || i >= left ? -1 : (b << 8) + i;
}

// Workgroup L's tile of a product over the groups' slots: units of `unit` slots, a.p.rtiles tiles
// of R each. Consecutive tiles of a group, in bands of 8 tiles of R, run on one XCD and share panels of both
// operands in its L2. With a.apart the units of at most unit / 2 slots run after all others.
// False past the last.
template <bool GATHER>
PMN_DEV bool group_tile(const GroupArgs& a, int64_t L, int64_t unit, FfnArgs& p, int64_t& trow, int64_t& tcol)
{
    const int64_t least = a.apart ? unit / 2 : 0;   // slots that a unit of the first ones has more than
    auto firsts = [=](int64_t n) { return (n + unit - 1 - least) / unit; };
    auto others = [=](int64_t n) { return (n + unit - 1) / unit - (n + unit - 1 - least) / unit; };
    const int64_t n = uniform64(group_units(a.offsets, a.G, firsts)) * a.p.rtiles, per = (n + 7) >> 3;
    const bool late = (L >> 3) >= per;
    if (late && !a.apart) return false;
    const int64_t i = late ? ffn_item_of(uniform64(group_units(a.offsets, a.G, others)) * a.p.rtiles, L - per * 8) : group_item_of(n, L);
    if (i < 0) return false;
    const int64_t u = i / a.p.rtiles;
    const GroupUnit w = late ? locate_group(a.offsets, a.G, u, others) : locate_group(a.offsets, a.G, u, firsts);
    if (w.g < 0) return false;
    const int64_t s0 = uniform64(w.s0), s1 = uniform64(w.s1), first = u - uniform64(w.index);
    group_at<GATHER>(a, __builtin_amdgcn_readfirstlane(w.g), s0, s1, p);
    p.ctiles = late ? 1 : firsts(s1 - s0);
    ffn_tile_at(p, i - first * a.p.rtiles, trow, tcol);
    if (late) tcol = firsts(s1 - s0);
    return true;
}

template <typename T, bool RKC, int EPI, bool GATHER>
__global__ __launch_bounds__(T::THREADS, T::RB * T::CB == 16 ? 1 : 2) void k_group_gemm(GroupArgs a)
{
    __shared__ __attribute__((aligned(1024))) uint8_t lds[T::LDS];
    if (T::RB * T::CB == 16) asm volatile("; agpr in use %0" ::"a"(0));   // keeps the 256 accumulators in AGPRs
    FfnArgs p;
    int64_t trow, tcol;
    if (!group_tile<GATHER>(a, blockIdx.x, T::BC, p, trow, tcol)) return;
    if constexpr (T::HALVES) {
        if (p.Nc - tcol * T::BC <= T::BC / 2) {
            ffn_tile<typename T::Half, RKC, true, EPI, GATHER ? GATHER_C : GATHER_NONE>(p, trow, 2 * tcol, 0, lds);
            return;
        }
    }
    ffn_tile<T, RKC, true, EPI, GATHER ? GATHER_C : GATHER_NONE>(p, trow, tcol, 0, lds);
}

// dW: p.Nr = K columns, p.Nc = N rows, contraction over the group's slots. The tiles of each group are
// dealt to all XCDs in runs, as the groups differ in length. With SPLIT the slots of each group go in a.splits
// parts (multiples of 32), whose sums stand one after another in p.out for k_group_wgrad_sum.
template <typename T, int EPI, bool GATHER, bool SPLIT>
__global__ __launch_bounds__(T::THREADS, T::RB * T::CB == 16 ? 1 : 2) void k_group_wgrad(GroupArgs a)
{
    __shared__ __attribute__((aligned(1024))) uint8_t lds[T::LDS];
    if (T::RB * T::CB == 16) asm volatile("; agpr in use %0" ::"a"(0));
    const int64_t tiles = a.p.rtiles * a.p.ctiles, per = (tiles + 7) >> 3;
    const int64_t j = blockIdx.x >> 3, gs = j / per, i = (blockIdx.x & 7) * per + (j - gs * per);
    if (i >= tiles || gs >= (SPLIT ? (int64_t)a.G * a.splits : a.G)) return;
    const int part = SPLIT ? (int)gs / a.G : 0;
    const int64_t g = SPLIT ? gs - (int64_t)part * a.G : gs;
    int64_t s0 = uniform64(a.offsets[g]), s1 = uniform64(a.offsets[g + 1]);
    if (SPLIT) {
        const int64_t n = s1 - s0, stages = (n + 31) >> 5, k1 = stages * (part + 1) / a.splits * 32;
        s1 = s0 + (k1 < n ? k1 : n);
        s0 += stages * part / a.splits * 32;
    }
    FfnArgs p = a.p;
    if (GATHER) p.gather += s0;
    else p.r += s0 * p.ldr;
    p.c += s0 * p.ldc;
    p.K = s1 - s0;
    p.out = static_cast<uint8_t*>(p.out) + gs * p.Nc * p.Nr * a.out_bytes;
    int64_t trow, tcol;
    ffn_tile_at(p, i, trow, tcol);
    ffn_tile<T, false, false, EPI, GATHER ? GATHER_R : GATHER_NONE>(p, trow, tcol, 0, lds);
}

// The parts' sums in their order, n8 times 8 values
template <bool F32>
__global__ __launch_bounds__(256) void k_group_wgrad_sum(const float* __restrict__ part, int splits, int64_t n8, void* __restrict__ out)
{
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n8) return;
    float v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    for (int s = 0; s < splits; s++) {
        const float4* q = reinterpret_cast<const float4*>(part + (s * n8 + i) * 8);
        const float4 a = q[0], b = q[1];
        v[0] += a.x; v[1] += a.y; v[2] += a.z; v[3] += a.w;
        v[4] += b.x; v[5] += b.y; v[6] += b.z; v[7] += b.w;
    }
    if (F32) {
        float4* dst = reinterpret_cast<float4*>(static_cast<float*>(out) + i * 8);
        dst[0] = make_float4(v[0], v[1], v[2], v[3]);
        dst[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + i * 8) =
            make_uint4(bf16x2_bits(v[0], v[1]), bf16x2_bits(v[2], v[3]), bf16x2_bits(v[4], v[5]), bf16x2_bits(v[6], v[7]));
    }
}

// Forward for few slots a group: units of 16 slots, the weights straight to registers. A workgroup holds
// 16 rows of W_g (SWIGLU: 8 features of w1 and the same of w3); its 8 wavefronts share the contraction
// in units of 64 k, one 128-byte line of each row, dealt in turn so that together they walk the rows, and
// their sums are added in order through LDS. Lanes past the unit's last slot repeat it and store nothing.
template <int EPI, bool GATHER>
__global__ __launch_bounds__(512, 2) void k_group_few(GroupArgs a)
{
    constexpr bool SWI = EPI == FFN_SWIGLU;
    constexpr int W = 8, U = 4;
    __shared__ float4 red[W][64];
    FfnArgs p;
    int64_t trow, tcol;
    if (!group_tile<GATHER>(a, blockIdx.x, 16, p, trow, tcol)) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int l16 = lane & 15, g = lane >> 4;
    const int64_t r0 = trow * (SWI ? 8 : 16), c = tcol * 16 + l16;
    const int64_t rows = SWI ? p.F : p.Nr;
    int64_t row = SWI ? r0 + (l16 & 7) : r0 + l16;
    row = row < rows ? row : rows - 1;
    if (SWI && l16 >= 8) row += p.F;
    const uint16_t* const rp = p.r + row * p.ldr + 8 * g;
    const int64_t slot = c < p.Nc ? c : p.Nc - 1;
    const uint16_t* const cp = p.c + (GATHER ? (int64_t)p.gather[slot] : slot) * p.ldc + 8 * g;
    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
    const int64_t units = p.K >> 6;
    auto load = [](const uint16_t* q) { return *reinterpret_cast<const bf16x8*>(q); };
    auto batch = [&](int64_t u, auto checked) {
        bf16x8 r[U][2], x[U][2];
#pragma unroll
        for (int i = 0; i < U; i++)
#pragma unroll
            for (int h = 0; h < 2; h++) {
                const int64_t k = (u + W * i) * 64 + 32 * h;
                if (!decltype(checked)::value || k + 8 * g < p.K) {
                    r[i][h] = load(rp + k);
                    x[i][h] = load(cp + k);
                } else {
                    r[i][h] = bf16x8{};
                    x[i][h] = bf16x8{};
                }
            }
#pragma unroll
        for (int i = 0; i < U; i++)
#pragma unroll
            for (int h = 0; h < 2; h++) acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(r[i][h], x[i][h], acc, 0, 0, 0);
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
    auto put = [](uint16_t* dst, const float (&o)[4]) {
        *reinterpret_cast<uint2*>(dst) = make_uint2(bf16x2_bits(o[0], o[1]), bf16x2_bits(o[2], o[3]));
    };
    if (SWI) {
        // lanes 0 .. 31 hold h1 of 8 features, lanes 32 .. 63 their h3
        float h3[4], o[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            h3[i] = __shfl_xor(v[i], 32, 64);
            o[i] = silu(v[i]) * h3[i];
        }
        const int64_t f = r0 + 4 * g;
        if (g >= 2 || c >= p.Nc || f >= p.F) return;
        put(static_cast<uint16_t*>(p.out) + c * p.F + f, o);
        if (p.out2) {
            put(p.out2 + c * 2 * p.F + f, v);
            put(p.out2 + c * 2 * p.F + p.F + f, h3);
        }
    } else {
        const int64_t n = r0 + 4 * g;
        if (c >= p.Nc || n >= p.Nr) return;
        if (EPI == FFN_F32) *reinterpret_cast<float4*>(static_cast<float*>(p.out) + c * p.Nr + n) = make_float4(v[0], v[1], v[2], v[3]);
        else put(static_cast<uint16_t*>(p.out) + c * p.Nr + n, v);
    }
}

typedef FfnTile<2, 2, 4, 4, 4> GroupLarge;   // 256 x 256, one workgroup per CU
typedef FfnTile<2, 2, 2, 2, 4> GroupMid;     // 128 x 128
typedef FfnTile<2, 2, 2, 1, 4> GroupSlim;    // 128 x 64

// Tiles and their times of one round of 256 workgroups, in us of a contraction of 4096 plus what a tile
// takes beside it (first loads, epilogue), taken from 60 sizes of 1 to 48 groups; half: a large tile of at most
// 128 slots, as nearly all are where the groups' mean is that small; alone: where there is no second round
// (two mid tiles fit a CU and slow each other).
struct GroupTile {
    int br, bc;
    double full, half, alone, rest;
};
enum { GROUP_LARGE = 0, GROUP_MID = 1, GROUP_SLIM = 2, GROUP_FEW = 3 };
static const GroupTile GROUP_TILES[4] = {{256, 256, 80.0, 52.0, 80.0, 14.0}, {128, 128, 43.0, 43.0, 33.0, 2.0},
                                         {128, 64, 29.5, 29.5, 23.0, 2.0}, {16, 16, 6.3, 6.3, 6.3, 1.0}};

// The tile whose rounds are shortest for a product of `rows` rows of R (contraction K) over M slots of G
// groups. The choice follows from the host's sizes: of the units that groups end in, half are taken to be one
// more each. (us, large / mid / slim / few: 480 slots in 48 groups of 4096 x 7168 465 / 464 / 496 / 663; 1024 in
// 4 of 4096 x 4096 77 / 52 / 81 / 482; 16 in 4 of 1024 x 7168 78 / 53 / 40 / 13.)
static int group_plan(int64_t M, int G, int64_t rows, int64_t K, bool rkc)
{
    const double some = (double)(M < G ? M : G);   // groups with slots, at most
    int best = GROUP_LARGE;
    double least = 0.0;
    for (int i = 0; i < (rkc ? 4 : 3); i++) {
        const GroupTile& t = GROUP_TILES[i];
        const double full = (double)((M + t.bc - 1) / t.bc) + (some - 1.0) / 2.0, units = full > some ? full : some;
        double rounds = units * (double)((rows + t.br - 1) / t.br) / 256.0;
        const double each = rounds <= 1.0 && t.alone < t.full ? t.alone : M <= 128 * some ? t.half : t.full;
        if (rounds <= 2.0) rounds = rounds <= 1.0 ? 1.0 : i == GROUP_MID ? rounds : 2.0;
        const double us = rounds * (each * (double)K / 4096.0 + t.rest);
        if (i == 0 || us < least) {
            best = i;
            least = us;
        }
    }
    return best;
}

// dW's tile: 256 x 256 (us of its rest beside the contraction: 8) or 128 x 128. (32 groups of 2048 x 4096,
// bf16: 512 slots 125 / 130, 8192 210 / 234, 131072 in fp32 1.76 / 2.1 ms; fewer than 256 large tiles leave CUs idle.)
static bool wgrad_large(int64_t M, int G, int64_t N, int64_t K)
{
    const double k = (double)M / G / 4096.0;
    auto us = [&](int b, double t, double rest) {
        const double rounds = (double)G * (double)((N + b - 1) / b) * (double)((K + b - 1) / b) / 256.0;
        return (rounds < 1.0 ? 1.0 : rounds) * (t * k + rest);
    };
    return us(256, 80.0, 8.0) <= us(128, 36.0, 2.0);
}

// Parts of each group's slots in wgrad, where the 128 x 128 tiles of all groups leave half of the CUs idle: a tile
// takes 36 us for 4096 slots, the parts are written and read at some 3 TB/s and their sum takes 5 us more; as many
// parts of 256 slots or more as make that least, if it gains 4 us. (With the data gradient: one
// group of 304 x 960 from 4767 slots 54 us in one part, 31 in seven; two of 512 x 1024 from 8192 51, 42 in four;
// without the bound two parts of 4 x 512 x 512 from 4096 slots took 23 us, one 21.)
static int wgrad_splits(int64_t M, int G, int64_t N, int64_t K)
{
    const int64_t tiles = G * ((N + 127) / 128) * ((K + 127) / 128);
    if (tiles > 128 || wgrad_large(M, G, N, K)) return 1;
    const double whole = (double)M / G * (36.0 / 4096.0), part = (double)(G * N * K) * 8.0 / 3e6;
    const int64_t most = M / G / 256 < 512 / tiles ? M / G / 256 : 512 / tiles;
    int best = 1;
    double least = whole - 4.0;
    for (int s = 2; s <= most && s <= 32; s++) {
        const double us = whole / s + s * part + 5.0;
        if (us < least) {
            best = s;
            least = us;
        }
    }
    return best;
}

size_t group_wgrad_part_bytes(int64_t M, int G, int64_t N, int64_t K)
{
    const int s = wgrad_splits(M, G, N, K);
    return s > 1 ? (size_t)s * G * N * K * 4 : 0;
}

// Workgroups of a product over the slots: rows of R in tiles of br, slots in units (a group adds at
// most one that is not full; two lists of them are dealt to the XCDs apart)
static int64_t group_grid(int64_t M, int G, int64_t rows, int64_t br, int64_t unit)
{
    const int64_t units = M / unit + G < M ? M / unit + G : M;
    return (units * ((rows + br - 1) / br) + 7) / 8 * 8 + 8;
}

static int64_t wgrad_grid(int G, int64_t N, int64_t K, int64_t b)
{
    return (((N + b - 1) / b) * ((K + b - 1) / b) + 7) / 8 * 8 * G;
}

// A launch has fewer than 2^32 threads.
constexpr int64_t MOST_THREADS = ((int64_t)1 << 32) - 1;

// The forward's launch, or dgrad's
bool group_rows_fit(int64_t M, int G, int64_t N, int64_t K, bool fwd)
{
    const GroupTile& t = GROUP_TILES[group_plan(M, G, fwd ? N : K, fwd ? K : N, fwd)];
    // (SwiGLU's F features in tiles of half as many are at most one tile of R more)
    return group_grid(M, G, fwd ? N : K, t.br, t.bc) + (M / t.bc + G) <= MOST_THREADS / (t.bc == 16 ? 512 : 256);
}

bool group_wgrad_fits(int64_t M, int G, int64_t N, int64_t K)
{
    return wgrad_grid(G, N, K, wgrad_large(M, G, N, K) ? 256 : 128) <= MOST_THREADS / 256;
}

template <typename T, bool RKC, int EPI, bool GATHER>
static void group_launch(GroupArgs a, int64_t M, hipStream_t stream)
{
    const int64_t nr = EPI == FFN_SWIGLU ? a.p.F : a.p.Nr, br = EPI == FFN_SWIGLU ? T::BR / 2 : T::BR;
    a.p.rtiles = (nr + br - 1) / br;
    // Where most units are half a one, the others go first: they take twice as long (2004 slots in 32 groups,
    // dgrad of 4096 x 1024: 137 us in the groups' order, 124 so; 4800 in 48 of 4096 x 7168: 624 / 593). Where
    // groups have many whole units, a half one reads again what the group's others had in L2 (24000 in 48:
    // 1461 / 1497).
    a.apart = T::HALVES && M <= T::BC / 2 * (M < a.G ? M : a.G);
    hipLaunchKernelGGL((k_group_gemm<T, RKC, EPI, GATHER>), dim3((unsigned)group_grid(M, a.G, nr, br, T::BC)), dim3(T::THREADS), 0,
                       stream, a);
}

template <bool RKC, int EPI, bool GATHER>
static void group_gemm(const GroupArgs& a, int64_t M, hipStream_t stream)
{
    const int plan = group_plan(M, a.G, a.p.Nr, a.p.K, RKC);
    if constexpr (RKC) {
        if (plan == GROUP_FEW) {
            GroupArgs b = a;
            const int64_t nr = EPI == FFN_SWIGLU ? a.p.F : a.p.Nr, br = EPI == FFN_SWIGLU ? 8 : 16;
            b.p.rtiles = (nr + br - 1) / br;
            hipLaunchKernelGGL((k_group_few<EPI, GATHER>), dim3((unsigned)group_grid(M, a.G, nr, br, 16)), dim3(512), 0, stream, b);
            return;
        }
    }
    if (plan == GROUP_LARGE) group_launch<GroupLarge, RKC, EPI, GATHER>(a, M, stream);
    else if (plan == GROUP_MID) group_launch<GroupMid, RKC, EPI, GATHER>(a, M, stream);
    else group_launch<GroupSlim, RKC, EPI, GATHER>(a, M, stream);
}

hipError_t launch_group_fwd_bf16(const uint16_t* x, const int32_t* gather, const uint16_t* w, const int64_t* offsets,
                                 int G, int64_t M, int64_t N, int64_t K, int epilogue, void* out, uint16_t* h13,
                                 hipStream_t stream)
{
    const bool swi = epilogue == PMN_EPI_SWIGLU, f32 = epilogue == PMN_EPI_F32;
    const int64_t F = N / 2;
    GroupArgs a{FfnArgs{w, x, K, K, N, 0, K, out, nullptr, swi ? h13 : nullptr, F}, offsets, G, N * K, swi ? F : N, f32 ? 4 : 2, N};
    a.p.gather = gather;
    if (gather) {
        if (swi) group_gemm<true, FFN_SWIGLU, true>(a, M, stream);
        else if (f32) group_gemm<true, FFN_F32, true>(a, M, stream);
        else group_gemm<true, FFN_BF16, true>(a, M, stream);
    } else {
        if (swi) group_gemm<true, FFN_SWIGLU, false>(a, M, stream);
        else if (f32) group_gemm<true, FFN_F32, false>(a, M, stream);
        else group_gemm<true, FFN_BF16, false>(a, M, stream);
    }
    return hipGetLastError();
}

// da (or with h13: dh13 [M x 2K], and a [M x K] where it is not null) and dw, each where not null; part: of
// group_wgrad_part_bytes
hipError_t launch_group_bwd_bf16(const uint16_t* dy, const uint16_t* x, const int32_t* gather, const uint16_t* w,
                                 const int64_t* offsets, int G, int64_t M, int64_t N, int64_t K, const uint16_t* h13,
                                 void* da, bool da_f32, uint16_t* act, void* dw, bool dw_f32, float* part,
                                 hipStream_t stream)
{
    if (da && M > 0) {
        GroupArgs a{FfnArgs{w, dy, K, N, K, 0, N, da, h13, act, K}, offsets, G, N * K, h13 ? 2 * K : K, da_f32 ? 4 : 2, K};
        if (h13) group_gemm<false, FFN_SWIGLU_BWD, false>(a, M, stream);
        else if (da_f32) group_gemm<false, FFN_F32, false>(a, M, stream);
        else group_gemm<false, FFN_BF16, false>(a, M, stream);
    }
    if (dw) {
        const int splits = wgrad_splits(M, G, N, K);
        const bool parts = splits > 1;
        GroupArgs a{FfnArgs{x, dy, K, N, K, N, 0, parts ? part : dw, nullptr, nullptr, 0}, offsets, G, 0, 0, parts || dw_f32 ? 4 : 2, 0};
        a.p.gather = gather;
        a.splits = splits;
        auto run = [&](auto tile, auto epi, auto split) {
            typedef decltype(tile) T;
            constexpr bool S = decltype(split)::value;
            a.p.rtiles = (K + T::BR - 1) / T::BR;
            a.p.ctiles = (N + T::BC - 1) / T::BC;
            const dim3 grid((unsigned)(wgrad_grid(G, N, K, T::BR) * splits)), block(T::THREADS);
            if (gather) hipLaunchKernelGGL((k_group_wgrad<T, decltype(epi)::value, true, S>), grid, block, 0, stream, a);
            else hipLaunchKernelGGL((k_group_wgrad<T, decltype(epi)::value, false, S>), grid, block, 0, stream, a);
        };
        typedef std::integral_constant<int, FFN_F32> F32;
        typedef std::integral_constant<int, FFN_BF16> BF16;
        if (wgrad_large(M, G, N, K)) {
            if (dw_f32) run(GroupLarge{}, F32{}, std::false_type{});
            else run(GroupLarge{}, BF16{}, std::false_type{});
        } else if (!parts) {
            if (dw_f32) run(GroupMid{}, F32{}, std::false_type{});
            else run(GroupMid{}, BF16{}, std::false_type{});
        } else {
            run(GroupMid{}, F32{}, std::true_type{});
            const int64_t n8 = G * N * K / 8;
            const dim3 grid((unsigned)((n8 + 255) / 256)), block(256);
            if (dw_f32) hipLaunchKernelGGL(k_group_wgrad_sum<true>, grid, block, 0, stream, part, splits, n8, dw);
            else hipLaunchKernelGGL(k_group_wgrad_sum<false>, grid, block, 0, stream, part, splits, n8, dw);
        }
    }
    return hipGetLastError();
}

}  // namespace pmn
