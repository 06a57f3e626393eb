// bf16_tile.hpp -- one tile of a bf16 product, shared by the dense feed-forward block (ffn.hip) and the
// products grouped by expert (gemm_bf16.hip).
//
// Every product is out[c, r] = sum_k R(r, k) C(c, k) on v_mfma_f32_32x32x16_bf16 with fp32
// accumulators. "R" supplies the accumulator's rows (columns of the output: an output row's values
// stand 4 in a lane), "C" its columns. An operand is either k-contiguous (KC: its stored rows are rows
// of the product) or row-contiguous (RC: stored transposed, one stored row per k: the weights in
// dgrad, both operands in wgrad).
//
// Operands stream through a ring of LDS stages of 32 k, filled by buffer_load ... lds (global -> LDS
// without registers), 1 KB pieces dealt evenly to the wavefronts, so "stage s has landed" is the
// per-wavefront condition vmcnt <= loads issued after it, followed by a barrier. A wavefront reads the
// fragments of stage v + 1 while the MFMAs of stage v run from registers. Bounds are the buffer
// descriptor's: rows and k past the operand read as zeros, so every size that is a multiple of 8 runs
// the same code.
//   KC stage: in the tiles with PAIRS, where both operands are KC or C alone is, two stages at a time: rows
//     of 128 bytes, 16-byte chunk c of row r at slot c ^ ((r / 2) % 8), so that a load takes whole lines of 8
//     rows and not halves of 16 (49152 x 4096 x 7168, both KC: 2130 us with halves, 2025 so; 65536 x 7168 x 2048
//     in 48 groups, C alone: 1866 and 1770). In the others (a split contraction's short parts) single stages:
//     rows of 64 bytes, chunk c at slot c ^ ((r / 4) % 4): a quarter wavefront's ds_read_b128 covers all 64
//     banks (248 B/clk/CU measured).
//   RC stage: 32 stored rows (k) of the tile's width, read by ds_read_b64_tr_b16, which hands lane i
//     of 16 the column i of 4 k; the 32-byte pairs of chunks of row k are permuted by
//     ((k / 8) % 2) | 2 (k % 4), so that the 4 k of 16 lanes lie in different banks (174 B/clk/CU
//     measured; 64 without).
//
// The accumulators leave through LDS, 32 output rows of a wavefront column at a time, so that a
// thread finishes 8 consecutive values of an output row with 16-byte accesses.
#pragma once

#include <type_traits>

#include "pmn_dev.hpp"

namespace pmn {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

enum { FFN_SWIGLU = 0, FFN_ADD = 1, FFN_SWIGLU_BWD = 2, FFN_BF16 = 3, FFN_F32 = 4, FFN_PART = 5 };

struct FfnArgs {
    const uint16_t* r;      // R operand, ldr elements between its stored rows
    const uint16_t* c;
    int64_t ldr, ldc;
    int64_t Nr, Nc, K;      // product: Nc output rows x Nr output columns, contraction K
    void* out;              // [Nc x Nr] (SWIGLU: a [Nc x F]; SWIGLU_BWD: dh13 [Nc x 2F])
    const uint16_t* aux;    // ADD: add (or null); SWIGLU_BWD: h13
    uint16_t* out2;         // SWIGLU: h13 (or null); SWIGLU_BWD: a (or null)
    int64_t F;
    float* part;            // PART: [splits x Nc x Nr]
    int splits;
    int64_t rtiles, ctiles;
    int64_t whole;          // tiles that run whole; the others in two halves (ffn_grid)
    const int32_t* gather;  // GATHER: the stored row that each row of C, or each k of R, is
};
enum { GATHER_NONE = 0, GATHER_C = 1, GATHER_R = 2 };

// The 16-byte words of aux that 8 consecutive outputs n .. n+7 of output row c need: ADD's add, or
// SWIGLU_BWD's h1 and h3.
template <int EPI>
PMN_DEV void ffn_aux8(const FfnArgs& p, int64_t c, int64_t n, uint4 (&w)[2])
{
    if (EPI == FFN_SWIGLU_BWD) {
        w[0] = *reinterpret_cast<const uint4*>(p.aux + c * 2 * p.F + n);
        w[1] = *reinterpret_cast<const uint4*>(p.aux + c * 2 * p.F + p.F + n);
    } else if (EPI == FFN_ADD) {
        w[0] = p.aux ? *reinterpret_cast<const uint4*>(p.aux + c * p.Nr + n) : make_uint4(0u, 0u, 0u, 0u);
    }
}

PMN_DEV void bf16x8_values(const uint4 w, float (&o)[8])
{
    const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int q = 0; q < 4; q++) {
        o[2 * q] = bf16_lo(a[q]);
        o[2 * q + 1] = bf16_hi(a[q]);
    }
}

// 8 consecutive outputs n .. n+7 of output row c from their fp32 sums (SWIGLU: v = h1, v2 = h3 of
// features n .. n+7) and their words of aux, read earlier by the same thread: out may be aux itself.
template <int EPI>
PMN_DEV void ffn_finish8(const FfnArgs& p, int64_t c, int64_t n, float (&v)[8], float (&v2)[8], const uint4 (&aux)[2])
{
    // LAST: not read again by this call, so stored past the caches
    auto put = [](uint16_t* dst, const float (&o)[8], bool last) {
        typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
        const u32x4 w = {bf16x2_bits(o[0], o[1]), bf16x2_bits(o[2], o[3]), bf16x2_bits(o[4], o[5]),
                         bf16x2_bits(o[6], o[7])};
        if (last) __builtin_nontemporal_store(w, reinterpret_cast<u32x4*>(dst));
        else *reinterpret_cast<u32x4*>(dst) = w;
    };
    if (EPI == FFN_SWIGLU) {
        float a[8];
#pragma unroll
        for (int u = 0; u < 8; u++) a[u] = silu(v[u]) * v2[u];
        put(static_cast<uint16_t*>(p.out) + c * p.F + n, a, false);
        if (p.out2) {
            put(p.out2 + c * 2 * p.F + n, v, true);
            put(p.out2 + c * 2 * p.F + p.F + n, v2, true);
        }
    } else if (EPI == FFN_SWIGLU_BWD) {
        float h1[8], h3[8], a[8];
        bf16x8_values(aux[0], h1);
        bf16x8_values(aux[1], h3);
#pragma unroll
        for (int u = 0; u < 8; u++) {
            // silu'(h) = s (1 + h (1 - s)); the values are rounded to bf16, far coarser than the
            // hardware exp2 and reciprocal
            const float s = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-h1[u] * 1.44269504088896341f));
            a[u] = h1[u] * s * h3[u];
            v2[u] = v[u] * h1[u] * s;
            v[u] = v[u] * h3[u] * (s * (1.0f + h1[u] * (1.0f - s)));
        }
        put(static_cast<uint16_t*>(p.out) + c * 2 * p.F + n, v, false);
        put(static_cast<uint16_t*>(p.out) + c * 2 * p.F + p.F + n, v2, false);
        if (p.out2) put(p.out2 + c * p.F + n, a, false);
    } else if (EPI == FFN_F32) {
        float4* dst = reinterpret_cast<float4*>(static_cast<float*>(p.out) + c * p.Nr + n);
        dst[0] = make_float4(v[0], v[1], v[2], v[3]);
        dst[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        if (EPI == FFN_ADD) {
            float b[8];
            bf16x8_values(aux[0], b);
#pragma unroll
            for (int u = 0; u < 8; u++) v[u] += b[u];
        }
        put(static_cast<uint16_t*>(p.out) + c * p.Nr + n, v, true);
    }
}

// 16 bytes per lane from buffer offset voff + soff (voff past the buffer: zeros) to LDS lds + 16 lane. The
// s_nop is the wait state that an LDS load needs after a write of m0.
PMN_DEV void dma16_buffer(i32x4 rsrc, uint32_t voff, uint32_t soff, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" ::"s"(lds), "v"(voff), "s"(rsrc), "s"(soff)
                 : "memory", "m0");
}

constexpr uint32_t FFN_OUTSIDE = 0x80000000u;   // a buffer offset past every descriptor

// The same from an address of the lane's own: rows that are gathered lie anywhere in 64 bits.
PMN_DEV void dma16_flat(const void* src, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds), "v"(src) : "memory", "m0");
}
static __device__ const uint4 ffn_zeros = {0u, 0u, 0u, 0u};   // what a gathered chunk outside the operand reads

// WR x WC wavefronts, each RB x CB blocks of 32 x 32; a ring of NST stages, or of two and a half or three pairs
// of them (PAIRS, where both operands are k-contiguous; where C alone is, NST stages of R and three pairs of C)
template <int WR_, int WC_, int RB_, int CB_, int NST_, bool PAIRS_ = true>
struct FfnTile {
    static constexpr int WR = WR_, WC = WC_, RB = RB_, CB = CB_, NST = NST_;
    static constexpr int BR = WR * RB * 32, BC = WC * CB * 32;
    static constexpr int THREADS = WR * WC * 64;
    static constexpr int RBYTES = BR * 64, STAGE = (BR + BC) * 64;
    static constexpr int RPW = BR / 16 / (WR * WC), CPW = BC / 16 / (WR * WC), PPW = RPW + CPW;   // pieces per wavefront
    static constexpr int OPITCH = BR + 4;                       // floats per staged output row
    static constexpr int OROWS = WC * 32;                       // output rows staged at a time
    static constexpr bool HALVES = RB_ * CB_ == 16;
    typedef FfnTile<WR_, WC_, RB_, CB_ / 2, NST_, PAIRS_> Half;   // of the output rows, all of the columns
    static constexpr bool PAIRS = PAIRS_;         // of stages, where an operand is k-contiguous
    static constexpr int RING = !PAIRS ? NST * STAGE : BR == BC ? 5 * BR * 128 : 3 * (BR + BC) * 128, OUTB = OROWS * OPITCH * 4;
    static constexpr int LDS = RING > OUTB ? RING : OUTB;
    static_assert(BR / 16 % (WR * WC) == 0 && BC / 16 % (WR * WC) == 0, "every wavefront loads the same pieces");
    static_assert(!PAIRS || RPW % 2 == 0, "half of a pair's pieces of R in each step");
    static_assert((PAIRS ? 6 : NST - 1) * (PPW + 1) <= 63, "vmcnt");   // loads on their way before the first wait
};

// Item number of workgroup L among n: workgroups L, L + 8, .. run on one XCD and take consecutive items.
// Negative past the last.
PMN_DEV int64_t ffn_item_of(int64_t n, int64_t L)
{
    const int64_t per = (n + 7) >> 3, i = (L & 7) * per + (L >> 3);
    return (L >> 3) >= per || i >= n ? -1 : i;
}

// Tile i of a product's rtiles x ctiles: in bands of 8 tile rows walked down their columns, so that the
// 32 tiles of an XCD at a time share 8 + 4 operand panels in its L2.
PMN_DEV void ffn_tile_at(const FfnArgs& p, int64_t i, int64_t& trow, int64_t& tcol)
{
    const int64_t band = i / (8 * p.ctiles), in = i - band * 8 * p.ctiles;
    const int64_t height = p.rtiles - band * 8 < 8 ? p.rtiles - band * 8 : 8;
    tcol = in / height;
    trow = band * 8 + (in - tcol * height);
}

// 4 bytes per lane to LDS lds + 4 lane
PMN_DEV void dma4_flat(const void* src, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(lds), "v"(src) : "memory", "m0");
}

// The tile (trow, tcol) of a product, or part `split` of its contraction (PART). GATHER_C: row i of C
// (k-contiguous) is stored row gather[i] of c. GATHER_R: k of R (row-contiguous) is stored row gather[k] of r.
template <typename T, bool RKC, bool CKC, int EPI, int GATHER = GATHER_NONE>
PMN_DEV void ffn_tile(const FfnArgs& p, int64_t trow, int64_t tcol, int split, uint8_t* lds)
{
    constexpr int BR = T::BR, BC = T::BC, RB = T::RB, CB = T::CB, PPW = T::PPW;
    constexpr bool SWI = EPI == FFN_SWIGLU, LINES = T::PAIRS && RKC && CKC;
    constexpr bool CLINES = T::PAIRS && CKC, ONE_PAIR = CLINES && !RKC;   // C alone by pairs of stages
    constexpr int NST = T::NST;
    constexpr int NR = LINES ? 2 * T::RPW : T::RPW, NC = CLINES ? 2 * T::CPW : T::CPW, NPC = NR + NC;   // pieces of a wavefront
    constexpr int PR = LINES ? 8 : 16, PC = CLINES ? 8 : 16;   // rows of a k-contiguous operand's piece
    constexpr int RSTEP = ONE_PAIR ? T::RBYTES : T::STAGE;       // bytes from a stage's R to the next one's
    static_assert(!ONE_PAIR || NST * T::RBYTES + 3 * BC * 128 <= T::LDS, "stages of R, pairs of C");
    static_assert(!SWI || (RB % 2 == 0 && RKC), "w1 and w3 rows of a feature stand in one wavefront");
    static_assert(GATHER != GATHER_C || CKC, "C's rows are gathered where it is k-contiguous");
    static_assert(GATHER != GATHER_R || (!RKC && !CKC && EPI != FFN_PART), "R's k are gathered where it is row-contiguous, in wgrad");
    // GATHER_R: the indices of a wavefront's rows of a stage, loaded 8 stages ahead into 8 slots behind the ring
    constexpr int ROWS = 512 / BR, SLOTS = 8, SLOT = 256;   // stored rows of a piece of R
    static_assert(GATHER != GATHER_R || (NST == 4 && T::RPW * ROWS == 8 && NST * T::STAGE + T::WR * T::WC * SLOTS * SLOT <= T::LDS), "index slots");
    constexpr int LPS = PPW + (GATHER == GATHER_R ? 1 : 0);   // loads of a stage and wavefront
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wr = wave / T::WC, wc = wave % T::WC, l32 = lane & 31, hh = lane >> 5;
    const int64_t r0 = trow * (SWI ? BR / 2 : BR), c0 = tcol * BC;
    const int64_t KT = (p.K + 31) >> 5;
    const int64_t s0 = EPI == FFN_PART ? KT * split / p.splits : 0;
    const int64_t s1 = EPI == FFN_PART ? KT * (split + 1) / p.splits : KT;
    const int nst = (int)(s1 - s0);

    // This wavefront's pieces, RPW of R and then CPW of C: byte offset of the lane's 16 bytes from the
    // operand's first at the stage, and for a k-contiguous operand the lane's first k of the stage.
    // Workgroups that share a panel start at different pieces of it, or they would ask one L2 channel for
    // the same lines at once: 4 to 5% at 128 x 128 (600 .. 2000 rows forward); 256 x 256 tiles are bound by
    // their MFMAs and run 1% slower with it.
    constexpr bool ROTATE = RB * CB < 16;
    const int rotr = ROTATE ? (int)(tcol % (BR / PR)) : 0, rotc = ROTATE ? (int)(trow % (BC / PC)) : 0;
    auto piece_of = [&](int i) {   // piece of its operand's tile
        return i < NR ? (wave * NR + i + rotr) % (BR / PR) : (wave * NC + i - NR + rotc) % (BC / PC);
    };
    uint32_t voff[NPC];
    int kch[NPC];
    const uint8_t* from[GATHER == GATHER_C ? NC : 1];   // the gathered rows' chunks at this part's first stage
#pragma unroll
    for (int i = 0; i < NPC; i++) {
        const bool isr = i < NR;
        const int q = piece_of(i);
        const int64_t ld = isr ? p.ldr : p.ldc;
        if (isr ? RKC : CKC) {
            const bool lines = isr ? LINES : CLINES;
            const int t = lines ? q * 8 + (lane >> 3) : q * 16 + (lane >> 2);   // tile row
            const int ch = lines ? (lane & 7) ^ ((t >> 1) & 7) : (lane & 3) ^ ((t >> 2) & 3);
            int row = t;                                              // from the tile's first
            bool ok;
            if (SWI && isr) {
                // features of w1 (blocks 0 .. RB / 2 - 1 of a wavefront) or w3 (the others)
                row = (t / (32 * RB)) * (16 * RB) + ((t >> 5) % (RB / 2)) * 32 + (t & 31);
                ok = r0 + row < p.F;
            } else {
                ok = (isr ? r0 : c0) + t < (isr ? p.Nr : p.Nc);
            }
            voff[i] = ok ? (uint32_t)(row * ld * 2 + ch * 16) : FFN_OUTSIDE;
            kch[i] = ch * 8;
            if (GATHER == GATHER_C && !isr) {
                from[i - NR] = ok ? reinterpret_cast<const uint8_t*>(p.c + (int64_t)p.gather[c0 + t] * ld + s0 * 32 + ch * 8)
                                      : nullptr;
                if (!ok) kch[i] = 0x7FFFFFFF;   // past every stage
            }
        } else {
            const int W = isr ? BR * 2 : BC * 2;                      // bytes of a stored row in the tile
            const int k = (q * 1024 + lane * 16) / W, ch = (q * 1024 + lane * 16) % W / 16;
            const int sw = ((k >> 3) & 1) | ((k & 3) << 1);
            const int col = ((((ch >> 1) ^ sw) << 1) | (ch & 1)) * 8;
            const bool ok = (isr ? r0 : c0) + col < (isr ? p.Nr : p.Nc);
            voff[i] = ok ? (uint32_t)(k * ld * 2 + col * 2) : FFN_OUTSIDE;
            kch[i] = 0;
            if (GATHER == GATHER_R && isr) {
                voff[i] = col * 2;              // within a stored row
                kch[i] = ok ? k : 0x7FFFFFFF;   // the lane's k of the stage
            }
        }
    }
    const uint32_t lds0 = (uint32_t)(uintptr_t)((__attribute__((address_space(3))) uint8_t*)lds);
    // A stage of this part: the operands' descriptors and how far it lies from the part's first. A
    // k-contiguous operand's descriptor stays, its stage is the offset `at`; it is bounded by the lanes' row
    // and chunk checks alone, which hold for its first row and no other (its own byte count as a second
    // bound took 10 to 30% of the forward, counted in 32 bits 1 to 4%). A row-contiguous one's begins at the
    // stage and ends with the contraction, or 32 rows past the stage.
    const int kend = (int)(p.K < s1 * 32 ? p.K : s1 * 32);
    const int64_t k0 = s0 * 32;
    struct Stage {
        uint64_t r, c;    // first bytes
        int rrec, crec;   // and bytes from there
        uint32_t at;
        int left;         // k from the stage's first to the part's end: none where it is not positive
        uint32_t dst, dstc;   // where R's and C's pieces go
        uint32_t atc;         // ONE_PAIR: at and left of C's pair
        int leftc;
    };
    const uint64_t r3 = SWI ? (uint64_t)p.F * p.ldr * 2 : 0;   // from w1's rows to w3's
    constexpr bool ONE_HALF = SWI && !ROTATE && RB % T::RPW == 0;   // a wavefront's pieces of R are all of w1 or all of w3
    auto of_w3 = [&](int i) { return SWI && ((piece_of(i) * PR) >> 5) % RB >= RB / 2; };
    auto records = [&](int left, int64_t ld, int64_t at) {
        const int rows = left < 64 ? left : 64;
        return rows > 0 ? (int)((rows * (int)ld - (int)at) * 2) : 0;
    };
    auto stage_at = [&](int s) {
        Stage g;
        g.r = GATHER == GATHER_R ? 0 : reinterpret_cast<uint64_t>(RKC ? p.r + r0 * p.ldr + k0 : p.r + (k0 + (int64_t)s * 32) * p.ldr + r0);
        if (ONE_HALF && of_w3(0)) g.r += r3;
        g.c = reinterpret_cast<uint64_t>(CKC ? p.c + c0 * p.ldc + k0 : p.c + (k0 + (int64_t)s * 32) * p.ldc + c0);
        g.at = (uint32_t)s * 64;
        g.left = kend - (int)k0 - s * 32;
        g.rrec = RKC ? 0x7FFFFFFF : records(g.left, p.ldr, r0);
        g.crec = CKC ? 0x7FFFFFFF : records(g.left, p.ldc, c0);
        g.dst = (uint32_t)(s % NST) * RSTEP + lds0;
        g.dstc = ONE_PAIR ? lds0 + NST * T::RBYTES : g.dst + T::RBYTES;
        g.atc = g.at;
        g.leftc = g.left;
        return g;
    };
    // the same `by` stages on; in scalar instructions few enough for the gap between two MFMAs
    auto advance = [&](Stage& g, auto by) {
        constexpr int BY = decltype(by)::value;
        g.left -= 32 * BY;
        g.at += 64 * BY;
        g.dst += BY * RSTEP;
        g.dst = g.dst >= lds0 + NST * RSTEP ? g.dst - NST * RSTEP : g.dst;
        if (!ONE_PAIR) g.dstc = g.dst + T::RBYTES;
        if (!RKC && GATHER != GATHER_R) {
            g.r += (uint64_t)(64 * BY) * p.ldr;
            g.rrec = records(g.left, p.ldr, r0);
        }
        if (!CKC) {
            g.c += (uint64_t)(64 * BY) * p.ldc;
            g.crec = records(g.left, p.ldc, c0);
        }
    };
    auto next_c = [&](Stage& g) {   // ONE_PAIR: C's next pair
        g.atc += 128;
        g.leftc -= 64;
        g.dstc = g.dstc == lds0 + NST * T::RBYTES + 2 * BC * 128 ? lds0 + NST * T::RBYTES : g.dstc + BC * 128;
    };
    auto descriptor = [](uint64_t first, int bytes) {
        return i32x4{__builtin_amdgcn_readfirstlane((int)(uint32_t)first), __builtin_amdgcn_readfirstlane((int)(uint32_t)(first >> 32)),
                     __builtin_amdgcn_readfirstlane(bytes), 0x00020000};
    };
    // Piece i's lane offset in stage g: chunks past the part's end of a k-contiguous operand lie outside
    auto lane_offset = [&](const Stage& g, int i) { return (i < NR ? RKC : CKC) && kch[i] >= (ONE_PAIR ? g.leftc : g.left) ? FFN_OUTSIDE : voff[i]; };
    struct Index {
        uint32_t v[GATHER == GATHER_R ? T::RPW : 1];
    };
    Index index;   // stored rows of this wavefront's pieces of R of the stage that is loaded next
    const int sub = (lane * 16) / (BR * 2);   // the lane's row of a piece
    const int64_t last = p.K > 0 ? p.K - 1 : 0;
    auto index_at = [&](int64_t k) { return p.K > 0 ? p.gather + (k < last ? k : last) : reinterpret_cast<const int32_t*>(&ffn_zeros); };
    const uint32_t slot0 = lds0 + NST * T::STAGE + wave * (SLOTS * SLOT);
    auto load_index = [&](int s) {   // lane e (of 8) of each 8: row e / RPW of piece e % RPW
        const int e = lane & 7;
        const int piece = (wave * T::RPW + e % T::RPW + rotr) % (BR / 16);
        dma4_flat(index_at((int64_t)s * 32 + piece * ROWS + e / T::RPW), slot0 + (s & (SLOTS - 1)) * SLOT);
    };
    auto read_index = [&](int s) {
        const uint32_t* a = reinterpret_cast<const uint32_t*>(lds + NST * T::STAGE + wave * (SLOTS * SLOT) + (s & (SLOTS - 1)) * SLOT) + sub * T::RPW;
        Index x;
#pragma unroll
        for (int i = 0; i < T::RPW; i++) x.v[GATHER == GATHER_R ? i : 0] = a[i];
        return x;
    };
    auto issue_piece = [&](const Stage& g, int i, uint32_t v) {
        const bool isr = i < NR;
        if (GATHER == GATHER_R && isr) {
            const uint8_t* z = reinterpret_cast<const uint8_t*>(&ffn_zeros);
            const uint8_t* row = reinterpret_cast<const uint8_t*>(p.r + r0) + (uint64_t)index.v[i] * (uint64_t)(uint32_t)(p.ldr * 2) + voff[i];
            dma16_flat(kch[i] >= g.left ? z : row, g.dst + piece_of(i) * 1024);
        } else if (GATHER == GATHER_C && !isr) {
            const uint8_t* z = reinterpret_cast<const uint8_t*>(&ffn_zeros);
            dma16_flat(kch[i] >= (ONE_PAIR ? g.leftc : g.left) ? z : from[i - NR] + (ONE_PAIR ? g.atc : g.at), g.dstc + piece_of(i) * 1024);
        } else if (!isr) {
            dma16_buffer(descriptor(g.c, g.crec), v, ONE_PAIR ? g.atc : CKC ? g.at : 0u, g.dstc + piece_of(i) * 1024);
        } else {
            dma16_buffer(descriptor(!ONE_HALF && of_w3(i) ? g.r + r3 : g.r, g.rrec), v, RKC ? g.at : 0u, g.dst + piece_of(i) * 1024);
        }
    };

    struct Frags {
        bf16x8 r[RB][2], c[CB][2];
    };
    // lane constants of the fragment reads
    const int swz = (l32 >> 2) & 3, swl = (l32 >> 1) & 7;
    const int g16 = lane >> 4, i16 = lane & 15, swt = (g16 >> 1) | ((i16 >> 2) << 1);
    auto read_frag = [&](const uint8_t* base, auto kc, auto lines, int width, int blk, int ks, int half) -> bf16x8 {
        if constexpr (decltype(lines)::value) {
            return *reinterpret_cast<const bf16x8*>(base + (blk * 32 + l32) * 128 + (((4 * half + 2 * ks + hh) ^ swl) << 4));
        } else if constexpr (decltype(kc)::value) {
            return *reinterpret_cast<const bf16x8*>(base + (blk * 32 + l32) * 64 + (((2 * ks + hh) ^ swz) << 4));
        } else {
            // columns 32 blk + 16 (g16 % 2) .., k = 16 ks + 8 (g16 / 2) + i16 / 4 and 4 further
            const int pair = (2 * blk + (g16 & 1)) ^ swt;
            const uint8_t* a = base + (16 * ks + 8 * (g16 >> 1) + (i16 >> 2)) * width + pair * 32 + (i16 & 3) * 8;
            const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)a);
            const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(a + 4 * width));
            return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        }
    };
    constexpr int NREAD = 2 * (RB + CB);   // fragments of a stage, in the order of their use
    struct Place {   // a stage's fragments
        const uint8_t *r, *c;
        int half;    // of its pair
    };
    uint32_t pair_in = NST * T::RBYTES;   // ONE_PAIR: the pair of C that is read
    auto place_of = [&](int s, int half) {
        return Place{lds + (s % NST) * RSTEP, ONE_PAIR ? lds + pair_in : lds + (s % NST) * RSTEP + T::RBYTES, half};
    };
    auto read_one = [&](const Place& at, int n, Frags& f) {
        const int ks = n / (RB + CB), b = n % (RB + CB);
        if (b < RB) f.r[b][ks] = read_frag(at.r, std::integral_constant<bool, RKC>{}, std::integral_constant<bool, LINES>{}, BR * 2, wr * RB + b, ks, at.half);
        else f.c[b - RB][ks] = read_frag(at.c, std::integral_constant<bool, CKC>{}, std::integral_constant<bool, CLINES>{}, BC * 2, wc * CB + b - RB, ks, at.half);
    };

    f32x16 acc[RB][CB];
#pragma unroll
    for (int i = 0; i < RB; i++)
#pragma unroll
        for (int j = 0; j < CB; j++)
#pragma unroll
            for (int v = 0; v < 16; v++) acc[i][j][v] = 0.0f;

    // The MFMAs of a step, each followed by what fits next to it (a wavefront has a SIMD to itself in the
    // 256 x 256 tiles and issues one instruction in 4 cycles, 7 next to an MFMA): its PPW loads spread over the
    // step, each with its lane offset ready one MFMA earlier; the fragment reads of stage `next` in the other
    // places of the first three quarters, so that the last have come back before the next step's barrier;
    // the next stages' scalars (other) at the end.
    constexpr int NM = 2 * RB * CB, NRQ = NM * 3 / 4;
    constexpr bool ROOMY = NM >= 2 * (NREAD / 2 + PPW);   // loads and reads have places of their own
    auto load_of = [](int q) { return (q + 1) * PPW / NM > q * PPW / NM ? q * PPW / NM : -1; };   // at most one a place where ROOMY
    auto compute = [&](const Place& next, const Frags& cur, Frags& nxt, auto ready, auto load, auto other) {
        int read = 0;
        uint32_t v[PPW];
#pragma unroll
        for (int q = 0; q < NM; q++) {
            const int ks = q / (RB * CB), i = (q / CB) % RB, j = q % CB;
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(cur.r[i][ks], cur.c[j][ks], acc[i][j], 0, 0, 0);
            if constexpr (ROOMY) {
                if (q + 1 < NM && load_of(q + 1) >= 0) v[load_of(q + 1)] = ready(load_of(q + 1));
                if (load_of(q) >= 0) load(load_of(q), v[load_of(q)]);
                else if (read < NREAD) read_one(next, read++, nxt);
            } else {
#pragma unroll
                for (int n = q * NREAD / NRQ; n < (q + 1) * NREAD / NRQ && n < NREAD; n++) read_one(next, n, nxt);
#pragma unroll
                for (int n = q * PPW / NM; n < (q + 1) * PPW / NM; n++) load(n, ready(n));
            }
            other(q);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    Frags f0, f1;
    auto read_first = [&](const Place& at) {
#pragma unroll
        for (int n = 0; n < NREAD; n++) read_one(at, n, f0);
    };
    const std::integral_constant<int, 1> one;
    constexpr int LATE = NM * 3 / 4;   // where the next stages' scalars are formed
    if constexpr (!LINES) {
        Stage g = stage_at(0);
        if constexpr (GATHER == GATHER_R) {
            Index at[NST];
#pragma unroll
            for (int s = 0; s < NST; s++)
#pragma unroll
                for (int i = 0; i < T::RPW; i++) at[s].v[i] = (uint32_t)*index_at(s * 32 + piece_of(i) * ROWS + sub);
#pragma unroll
            for (int s = 0; s < NST; s++) {
                index = at[s];
#pragma unroll
                for (int i = 0; i < PPW; i++) issue_piece(g, i, lane_offset(g, i));
                load_index(s + NST);
                advance(g, one);
            }
        } else if constexpr (ONE_PAIR) {
            // R of stages 0 .. 3; C of pairs 0 and 1 and half of 2, as the steps before the first would load them
            static_assert(NST == 4, "three steps and a half ahead");
#pragma unroll
            for (int s = 0; s < NST; s++) {
#pragma unroll
                for (int i = 0; i < NR; i++) issue_piece(g, i, lane_offset(g, i));
                const int c0 = s == 2 ? NC / 2 : 0, c1 = s == 0 || s == 2 ? NC : NC / 2;
#pragma unroll
                for (int i = c0; i < c1; i++) issue_piece(g, NR + i, lane_offset(g, NR + i));
                if (s == 0 || s == 2) next_c(g);
                advance(g, one);
            }
        } else {
#pragma unroll
            for (int s = 0; s < NST; s++) {
#pragma unroll
                for (int i = 0; i < PPW; i++) issue_piece(g, i, lane_offset(g, i));
                advance(g, one);
            }
        }
        wait_loads_and_barrier<(NST - 1) * LPS>();
        read_first(place_of(0, 0));
        if constexpr (GATHER == GATHER_R) index = read_index(NST);
        // stage v + 1 has landed and every wavefront is done reading stage v, whose slot is refilled
        // (ONE_PAIR: an even step loads half of C's pair v / 2 + 2, an odd one half of the one after it, whose slot's
        // last fragments were read in the step before)
        auto step = [&](int v, auto second, const Frags& cur, Frags& nxt) {
            constexpr bool odd = decltype(second)::value;
            auto piece = [](int n) { return !ONE_PAIR || n < NR ? n : n + (odd ? 0 : NC / 2); };
            wait_loads_and_barrier<(NST - 2) * LPS>();
            const Stage h = g;   // stage v + NST
            Index ahead;
            if constexpr (GATHER == GATHER_R) ahead = read_index(v + NST + 1);
            if (ONE_PAIR && odd) pair_in = pair_in == NST * T::RBYTES + 2 * BC * 128 ? NST * T::RBYTES : pair_in + BC * 128;
            compute(place_of(v + 1, odd ? 0 : 1), cur, nxt, [&](int n) { return lane_offset(h, piece(n)); },
                    [&](int n, uint32_t o) { issue_piece(h, piece(n), o); },
                    [&](int q) {
                        if (q == LATE) advance(g, one);
                        if (ONE_PAIR && !odd && q == LATE) next_c(g);
                        if constexpr (GATHER == GATHER_R)
                            if (q == LATE + 1) load_index(v + 2 * NST);
                    });
            if constexpr (GATHER == GATHER_R) index = ahead;
        };
        for (int v = 0; v < nst; v += 2) {     // past an odd count the second step multiplies zeros
            step(v, std::false_type{}, f0, f1);
            step(v + 1, std::true_type{}, f1, f0);
        }
    } else {
        // Both operands k-contiguous: a row gives 64 bytes to a stage, half a 128-byte line. Stages go in
        // pairs, and a piece is 8 rows of a pair, whole lines. Pair p's first stage is multiplied while the
        // fragments of its second are read (its even step), its second while those of pair p + 1's first are
        // (its odd step), so that its slots are free from its odd step on. LDS holds two and a half pairs of
        // equal operands, as slots of one operand of a pair: R of pair p + 2 is loaded in the even step and C of
        // it in the odd one; or three pairs: half of pair p + 2's pieces, then half of pair p + 3's. (8192 x 7168 x 2048
        // forward: 707 us with single stages, 660 with pairs of half lines; halves to whole lines as above. A second
        // barrier, before the even step, changes nothing. Row-contiguous operands, whose stages are whole lines,
        // lose 5% by pairs.)
        constexpr bool EQUAL = BR == BC;
        constexpr uint32_t RPB = BR * 128, CPB = BC * 128, RING = EQUAL ? 5 * RPB : 3 * (RPB + CPB);
        struct At {
            uint32_t r, c;
        };
        auto next_pair = [](At& a) {
            if (EQUAL) {
                a.r = a.r >= 3 * RPB ? a.r - 3 * RPB : a.r + 2 * RPB;
                a.c = a.c >= 3 * RPB ? a.c - 3 * RPB : a.c + 2 * RPB;
            } else {
                a.r = a.r + RPB + CPB == RING ? 0 : a.r + RPB + CPB;
                a.c = a.r + RPB;
            }
        };
        At to{0, RPB}, in{0, RPB};
        Stage g = stage_at(0);
        g.dst = lds0 + to.r;
        g.dstc = lds0 + to.c;
        auto next_loads = [&] {
            next_pair(to);
            g.left -= 64;
            g.at += 128;
            g.dst = lds0 + to.r;
            g.dstc = lds0 + to.c;
        };
        // piece n of those that a step loads
        auto piece = [](int n, bool odd) {
            if (EQUAL) return odd ? NR + n : n;
            const int h = odd ? 0 : 1;
            return n < NR / 2 ? h * (NR / 2) + n : NR + h * (NC / 2) + n - NR / 2;
        };
#pragma unroll
        for (int s = 0; s < 2; s++) {
#pragma unroll
            for (int i = 0; i < NPC; i++) issue_piece(g, i, lane_offset(g, i));
            next_loads();
        }
        if (!EQUAL) {
#pragma unroll
            for (int i = 0; i < PPW; i++) issue_piece(g, piece(i, true), lane_offset(g, piece(i, true)));
        }
        wait_loads_and_barrier<EQUAL ? NPC : NPC + PPW>();
        auto stage_in = [&](int half) { return Place{lds + in.r, lds + in.c, half}; };
        read_first(stage_in(0));
        auto step = [&](auto second, const Frags& cur, Frags& nxt) {
            constexpr bool odd = decltype(second)::value;
            compute(stage_in(odd ? 0 : 1), cur, nxt, [&](int n) { return lane_offset(g, piece(n, odd)); },
                    [&](int n, uint32_t o) { issue_piece(g, piece(n, odd), o); }, [](int) {});
        };
        for (int v = 0; v < nst; v += 2) {
            step(std::false_type{}, f0, f1);
            next_pair(in);
            if (!EQUAL) next_loads();
            wait_loads_and_barrier<EQUAL ? NR : NPC>();   // pair p + 1 has landed
            step(std::true_type{}, f1, f0);
            if (EQUAL) next_loads();
        }
    }
    wait_loads_and_barrier<0>();

    // output rows c0 + wc * 32 CB + j * 32 .., staged as fp32 [WC * 32][BR]; a thread finishes NPC pieces
    // of 8 values, whose words of aux are on their way while the rows are staged
    float* const ot = reinterpret_cast<float*>(lds);
    constexpr int NW = (SWI ? BR / 2 : BR) / 8, NP = T::OROWS * NW / T::THREADS;
    static_assert(T::OROWS * NW % T::THREADS == 0, "whole pieces per thread");
    auto place = [&](int j, int k, int& rr, int& n, int64_t& c) {
        const int at = k * T::THREADS + tid;
        rr = at / NW;
        n = (at % NW) * 8;
        c = c0 + (rr >> 5) * (32 * CB) + j * 32 + (rr & 31);
        return c < p.Nc && r0 + n < (SWI ? p.F : p.Nr);
    };
    // The words of aux of the first AHEAD phases are asked for at once, the others' that many phases
    // before their use: as many as the registers hold that the fragments no longer need (8192 x 7168 x
    // 2048 forward: 660 us with one phase ahead, 621 with all four).
    constexpr bool AUX = EPI == FFN_ADD || EPI == FFN_SWIGLU_BWD;
    constexpr int AHEAD = EPI == FFN_ADD ? CB : 2;
    uint4 aux[CB][NP][2];
    auto load_aux = [&](int j) {
#pragma unroll
        for (int k = 0; k < NP; k++) {
            int rr, n;
            int64_t c;
            if (place(j, k, rr, n, c)) ffn_aux8<EPI>(p, c, r0 + n, aux[j][k]);
        }
    };
    if (AUX) {
#pragma unroll
        for (int j = 0; j < AHEAD && j < CB; j++) load_aux(j);
    }
#pragma unroll
    for (int j = 0; j < CB; j++) {
        if (AUX && j > 0 && j - 1 + AHEAD < CB) load_aux(j - 1 + AHEAD);
        if (j > 0) __syncthreads();
        float* const row = ot + (wc * 32 + l32) * T::OPITCH;
#pragma unroll
        for (int i = 0; i < RB; i++) {
            // SWIGLU: h1 in the first half of the row, h3 in the second
            const int n = SWI ? (i / (RB / 2)) * (BR / 2) + wr * 16 * RB + (i % (RB / 2)) * 32 : (wr * RB + i) * 32;
#pragma unroll
            for (int q = 0; q < 4; q++)
                *reinterpret_cast<float4*>(row + n + q * 8 + hh * 4) =
                    make_float4(acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]);
            __builtin_amdgcn_sched_barrier(0);
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < NP; k++) {
            int rr, n;
            int64_t c;
            if constexpr (EPI == FFN_F32) {
                // 4 values of each half of the tile's row: whole 128-byte lines of a row at a store
                typedef float f32x4u __attribute__((ext_vector_type(4)));
                place(j, k, rr, n, c);
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    const int m = h * (BR / 2) + n / 2;
                    if (c < p.Nc && r0 + m < p.Nr)
                        __builtin_nontemporal_store(*reinterpret_cast<const f32x4u*>(ot + rr * T::OPITCH + m),
                                                    reinterpret_cast<f32x4u*>(static_cast<float*>(p.out) + c * p.Nr + r0 + m));
                }
                continue;
            }
            if (!place(j, k, rr, n, c)) continue;
            const float* src = ot + rr * T::OPITCH + n;
            float v[8], v2[8];
#pragma unroll
            for (int u = 0; u < 8; u += 4) {
                const float4 a = *reinterpret_cast<const float4*>(src + u);
                v[u] = a.x; v[u + 1] = a.y; v[u + 2] = a.z; v[u + 3] = a.w;
                if (SWI) {
                    const float4 b = *reinterpret_cast<const float4*>(src + BR / 2 + u);
                    v2[u] = b.x; v2[u + 1] = b.y; v2[u + 2] = b.z; v2[u + 3] = b.w;
                }
            }
            if constexpr (EPI == FFN_PART) {
                float4* dst = reinterpret_cast<float4*>(p.part + ((int64_t)split * p.Nc + c) * p.Nr + r0 + n);
                dst[0] = make_float4(v[0], v[1], v[2], v[3]);
                dst[1] = make_float4(v[4], v[5], v[6], v[7]);
            } else {
                ffn_finish8<EPI>(p, c, r0 + n, v, v2, aux[j][k]);
            }
        }
    }
}

}  // namespace pmn
