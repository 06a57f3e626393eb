// ffn.hip -- the dense gated feed-forward block (the shared expert beside the routed ones) in bf16:
//     [h1 | h3] = x w13^T,  a = silu(h1) h3,  y = a w2^T (+ add)
// and its backward
//     da = dy w2,  dh1 = da h3 silu'(h1),  dh3 = da silu(h1)
//     dx = [dh1 | dh3] w13,  dw13 = [dh1 | dh3]^T x,  dw2 = dy^T a
// x, y, dy [M x H], w13 [2F x H] (w1 over w3), w2 [H x F], h13 [M x 2F], all row-major.
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
//   KC stage: rows of 64 bytes, 16-byte chunk c of row r at slot c ^ ((r / 4) % 4): a quarter
//     wavefront's ds_read_b128 covers all 64 banks (248 B/clk/CU measured).
//   RC stage: 32 stored rows (k) of the tile's width, read by ds_read_b64_tr_b16, which hands lane i
//     of 16 the column i of 4 k; the 32-byte pairs of chunks of row k are permuted by
//     ((k / 8) % 2) | 2 (k % 4), so that the 4 k of 16 lanes lie in different banks (174 B/clk/CU
//     measured; 64 without).
//
// a and dh13 are rounded to bf16 between the products, whose operands the bf16 MFMAs take (at most
// 2^-8 of a value; a second MFMA for what is rounded off would double those products): y and the gradients are
// off by 0.0021 to 0.0024 in norm, of which the rounding of the outputs themselves is 0.0017. h13 is stored
// in bf16; the forward's own a comes from the fp32 sums.
//
// The accumulators leave through LDS, 32 output rows of a wavefront column at a time, so that a
// thread finishes 8 consecutive values of an output row with 16-byte accesses. Where the tiles of a
// product are fewer than the compute units the contraction is split: the parts write fp32 sums and a
// second kernel adds them in order and finishes the rows, so results do not depend on the launch.
#include <type_traits>

#include "pmn_dev.hpp"
#include "pmn_kernels.hpp"

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
    uint16_t* out2;         // SWIGLU: h13 (or null); SWIGLU_BWD: a
    int64_t F;
    float* part;            // PART: [splits x Nc x Nr]
    int splits;
    int64_t rtiles, ctiles;
    int64_t whole;          // tiles that run whole; the others in two halves (ffn_grid)
};

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
        put(p.out2 + c * p.F + n, a, false);
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

// buffer descriptor of `bytes` bytes (at most 2^31 - 1) from p: loads past them return zero
PMN_DEV i32x4 buffer_of(const void* p, int64_t bytes)
{
    const uint64_t a = reinterpret_cast<uint64_t>(p);
    const int n = bytes < 0 ? 0 : (bytes > 0x7FFFFFFF ? 0x7FFFFFFF : (int)bytes);
    return i32x4{__builtin_amdgcn_readfirstlane((int)(uint32_t)a), __builtin_amdgcn_readfirstlane((int)(uint32_t)(a >> 32)),
                 __builtin_amdgcn_readfirstlane(n), 0x00020000};
}

// 16 bytes per lane from buffer offset voff (past the buffer: zeros) to LDS lds + 16 lane. The
// s_nop is the wait state that an LDS load needs after a write of m0.
PMN_DEV void dma16_buffer(i32x4 rsrc, uint32_t voff, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(lds), "v"(voff), "s"(rsrc)
                 : "memory", "m0");
}

constexpr uint32_t FFN_OUTSIDE = 0x80000000u;   // a buffer offset past every descriptor

// WR x WC wavefronts, each RB x CB blocks of 32 x 32; a ring of NST stages, or of 5 filled in pairs
template <int WR_, int WC_, int RB_, int CB_, int NST_>
struct FfnTile {
    static constexpr int WR = WR_, WC = WC_, RB = RB_, CB = CB_, NST = NST_;
    static constexpr int BR = WR * RB * 32, BC = WC * CB * 32;
    static constexpr int THREADS = WR * WC * 64;
    static constexpr int RBYTES = BR * 64, STAGE = (BR + BC) * 64;
    static constexpr int RPW = BR / 16 / (WR * WC), CPW = BC / 16 / (WR * WC), PPW = RPW + CPW;   // pieces per wavefront
    static constexpr int OPITCH = BR + 4;                       // floats per staged output row
    static constexpr int OROWS = WC * 32;                       // output rows staged at a time
    static constexpr bool HALVES = RB_ * CB_ == 16;
    typedef FfnTile<WR_, WC_, RB_, CB_ / 2, NST_> Half;         // of the output rows, all of the columns
    static constexpr bool PAIRS = RPW % 2 == 0 && CPW % 2 == 0;
    static constexpr int RING = (PAIRS ? 5 : NST) * STAGE, OUTB = OROWS * OPITCH * 4;
    static constexpr int LDS = RING > OUTB ? RING : OUTB;
    static_assert(BR / 16 % (WR * WC) == 0 && BC / 16 % (WR * WC) == 0, "every wavefront loads the same pieces");
    static_assert((PAIRS ? 6 : NST - 1) * PPW <= 63, "vmcnt");
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

// The tile (trow, tcol) of a product, or part `split` of its contraction (PART).
template <typename T, bool RKC, bool CKC, int EPI>
PMN_DEV void ffn_tile(const FfnArgs& p, int64_t trow, int64_t tcol, int split, uint8_t* lds)
{
    constexpr int BR = T::BR, BC = T::BC, RB = T::RB, CB = T::CB, PPW = T::PPW;
    constexpr bool SWI = EPI == FFN_SWIGLU, PAIRED = T::PAIRS && RKC && CKC;
    constexpr int NST = PAIRED ? 5 : T::NST;
    static_assert(!SWI || (RB % 2 == 0 && RKC), "w1 and w3 rows of a feature stand in one wavefront");
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
    const int rotr = ROTATE ? (int)(tcol % (BR / 16)) : 0, rotc = ROTATE ? (int)(trow % (BC / 16)) : 0;
    auto piece_of = [&](int i) {   // piece of its operand's tile
        return i < T::RPW ? (wave * T::RPW + i + rotr) % (BR / 16) : (wave * T::CPW + i - T::RPW + rotc) % (BC / 16);
    };
    uint32_t voff[PPW];
    int kch[PPW];
#pragma unroll
    for (int i = 0; i < PPW; i++) {
        const bool isr = i < T::RPW;
        const int q = piece_of(i);
        const int64_t ld = isr ? p.ldr : p.ldc;
        if (isr ? RKC : CKC) {
            const int t = q * 16 + (lane >> 2);                       // tile row
            const int ch = (lane & 3) ^ ((t >> 2) & 3);
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
        } else {
            const int W = isr ? BR * 2 : BC * 2;                      // bytes of a stored row in the tile
            const int k = (q * 1024 + lane * 16) / W, ch = (q * 1024 + lane * 16) % W / 16;
            const int sw = ((k >> 3) & 1) | ((k & 3) << 1);
            const int col = ((((ch >> 1) ^ sw) << 1) | (ch & 1)) * 8;
            const bool ok = (isr ? r0 : c0) + col < (isr ? p.Nr : p.Nc);
            voff[i] = ok ? (uint32_t)(k * ld * 2 + col * 2) : FFN_OUTSIDE;
            kch[i] = 0;
        }
    }
    const uint32_t lds0 = (uint32_t)(uintptr_t)((__attribute__((address_space(3))) uint8_t*)lds);
    // An operand's bytes from its first at stage 0 of this part, a stage's advance and how many bytes
    // there are. A k-contiguous operand is bounded by the lanes' row and chunk checks alone, which hold for
    // this base and no other: its own byte count as a second bound took 10 to 30% of the forward, counted
    // in 32 bits 1 to 4%.
    struct Operand {
        const uint8_t* base;
        int64_t step, bytes;
    };
    auto operand = [&](const uint16_t* src, bool kc, int64_t ld, int64_t at) {
        const int64_t k0 = s0 * 32;
        Operand o;
        o.base = reinterpret_cast<const uint8_t*>(kc ? src + at * ld + k0 : src + k0 * ld + at);
        o.step = kc ? 64 : 64 * ld;
        o.bytes = kc ? INT64_MAX : ((p.K - k0) * ld - at) * 2;
        return o;
    };
    const Operand opr = operand(p.r, RKC, p.ldr, r0), opc = operand(p.c, CKC, p.ldc, c0);
    const int64_t w3_bytes = SWI ? p.F * p.ldr * 2 : 0;
    struct Stage {
        i32x4 r, r3, c;   // r3: the rows of w3
        int left;         // k of this stage, at most 32
        uint32_t dst;
    };
    auto stage_at = [&](int s) {
        Stage g;
        const bool in = s < nst;   // nothing past the part's last stage
        g.r = buffer_of(opr.base + s * opr.step, in ? opr.bytes - s * opr.step : 0);
        if (SWI) g.r3 = buffer_of(opr.base + w3_bytes + s * opr.step, in ? opr.bytes - s * opr.step : 0);
        g.c = buffer_of(opc.base + s * opc.step, in ? opc.bytes - s * opc.step : 0);
        const int64_t left = p.K - (s0 + s) * 32;
        g.left = left > 32 ? 32 : (int)left;
        g.dst = (uint32_t)(s % NST) * T::STAGE;
        return g;
    };
    auto issue_piece = [&](const Stage& g, int i) {
        const bool isr = i < T::RPW;
        // chunks past K of a k-contiguous operand
        const uint32_t v = (isr ? RKC : CKC) && kch[i] >= g.left ? FFN_OUTSIDE : voff[i];
        if (!isr) {
            dma16_buffer(g.c, v, g.dst + lds0 + T::RBYTES + piece_of(i) * 1024);
        } else if (!SWI) {
            dma16_buffer(g.r, v, g.dst + lds0 + piece_of(i) * 1024);
        } else {
            const bool w3 = (piece_of(i) >> 1) % RB >= RB / 2;
            i32x4 d;
#pragma unroll
            for (int q = 0; q < 4; q++) d[q] = __builtin_amdgcn_readfirstlane(w3 ? g.r3[q] : g.r[q]);
            dma16_buffer(d, v, g.dst + lds0 + piece_of(i) * 1024);
        }
    };

    struct Frags {
        bf16x8 r[RB][2], c[CB][2];
    };
    // lane constants of the fragment reads
    const int swz = (l32 >> 2) & 3;
    const int g16 = lane >> 4, i16 = lane & 15, swt = (g16 >> 1) | ((i16 >> 2) << 1);
    auto read_frag = [&](const uint8_t* base, auto kc, int width, int blk, int ks) -> bf16x8 {
        if constexpr (decltype(kc)::value) {
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
    auto read_one = [&](const uint8_t* base, int n, Frags& f) {
        const int ks = n / (RB + CB), b = n % (RB + CB);
        if (b < RB) f.r[b][ks] = read_frag(base, std::integral_constant<bool, RKC>{}, BR * 2, wr * RB + b, ks);
        else f.c[b - RB][ks] = read_frag(base + T::RBYTES, std::integral_constant<bool, CKC>{}, BC * 2, wc * CB + b - RB, ks);
    };

    f32x16 acc[RB][CB];
#pragma unroll
    for (int i = 0; i < RB; i++)
#pragma unroll
        for (int j = 0; j < CB; j++)
#pragma unroll
            for (int v = 0; v < 16; v++) acc[i][j][v] = 0.0f;

    // The MFMAs of a step with its PPW loads spread over them and the fragment reads of stage `next`
    // over the first three quarters, so that the last have come back before the next step's barrier
    // (all loads before all reads measured 4% slower).
    constexpr int NM = 2 * RB * CB, NRQ = NM * 3 / 4;
    auto compute = [&](int next, const Frags& cur, Frags& nxt, auto load) {
        const uint8_t* rbase = lds + (next % NST) * T::STAGE;
#pragma unroll
        for (int q = 0; q < NM; q++) {
            const int ks = q / (RB * CB), i = (q / CB) % RB, j = q % CB;
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(cur.r[i][ks], cur.c[j][ks], acc[i][j], 0, 0, 0);
#pragma unroll
            for (int n = q * NREAD / NRQ; n < (q + 1) * NREAD / NRQ && n < NREAD; n++) read_one(rbase, n, nxt);
#pragma unroll
            for (int n = q * PPW / NM; n < (q + 1) * PPW / NM; n++) load(n);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    Frags f0, f1;
    auto read_first = [&] {
#pragma unroll
        for (int n = 0; n < NREAD; n++) read_one(lds, n, f0);
    };
    if constexpr (!PAIRED) {
#pragma unroll
        for (int s = 0; s < NST; s++) {
            const Stage g = stage_at(s);
#pragma unroll
            for (int i = 0; i < PPW; i++) issue_piece(g, i);
        }
        wait_loads_and_barrier<(NST - 1) * PPW>();
        read_first();
        // stage v + 1 has landed and every wavefront is done reading stage v, whose slot is refilled
        auto step = [&](int v, const Frags& cur, Frags& nxt) {
            wait_loads_and_barrier<(NST - 2) * PPW>();
            const Stage g = stage_at(v + NST);
            compute(v + 1, cur, nxt, [&](int n) { issue_piece(g, n); });
        };
        for (int v = 0; v < nst; v += 2) {     // past an odd count the second step multiplies zeros
            step(v, f0, f1);
            step(v + 1, f1, f0);
        }
    } else {
        // Both operands k-contiguous: a row gives 64 bytes to a stage, half a 128-byte line. Stages go in
        // pairs v, v + 1 (v even): a piece is loaded for both stages back to back, so that the second half
        // of its lines is in the first-level cache (8192 x 7168 x 2048 forward: 707 us with single stages,
        // 660 in pairs; row-contiguous operands, whose stages are whole lines, lose 5% by it). Slots of
        // stages v - 1 and v are free at step v; half of the pieces are loaded then, half at step v + 1.
#pragma unroll
        for (int s = 0; s < NST - 1; s += 2) {
            const Stage g0 = stage_at(s), g1 = stage_at(s + 1);
#pragma unroll
            for (int i = 0; i < PPW; i++) {
                issue_piece(g0, i);
                issue_piece(g1, i);
            }
        }
        wait_loads_and_barrier<(NST - 3) * PPW>();
        read_first();
        auto step = [&](int v, int odd, const Frags& cur, Frags& nxt) {
            const Stage g0 = stage_at(v + NST - 1), g1 = stage_at(v + NST);
            compute(v + odd + 1, cur, nxt, [&](int n) {
                const bool isr = n < T::RPW;
                const int m = isr ? n : n - T::RPW, half = (isr ? T::RPW : T::CPW) / 2;
                issue_piece(m & 1 ? g1 : g0, (isr ? 0 : T::RPW) + odd * half + (m >> 1));
            });
        };
        for (int v = 0; v < nst; v += 2) {
            wait_loads_and_barrier<63>();      // stage v + 1 landed with its pair
            step(v, 0, f0, f1);
            wait_loads_and_barrier<PPW>();     // the pair v + 2, v + 3: all but step v's loads
            step(v, 1, f1, f0);
        }
    }
    wait_loads_and_barrier<0>();

    // output rows c0 + wc * 32 CB + j * 32 .., staged as fp32 [WC * 32][BR]; a thread finishes NP pieces
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
    else if constexpr (CKC) ffn_launch_tile<FfnFew, RKC, CKC, FFN_PART>(p, stream);
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
