// adamw.hip -- one AdamW step over many tensors in one launch, with states in fp32 or in 8 bits.
//
// Per value, with g' = grad_scale * g and t the step (from 1):
//     m = b1 m + (1 - b1) g',   v = b2 v + (1 - b2) g'^2
//     p = p (1 - lr wd) - lr (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps)
// and a bf16 copy of p for the quantizers and GEMMs.
// In 8 bits m is kept as MXFP8 (E4M3 codes, one E8M0 per 32 values) and v as the MXFP8 of sqrt(v):
// the root halves the exponent range, so a block's E4M3 codes reach 2^-17 of its largest root, 2^-34
// of its largest v. Both round stochastically (the requant's rule and its index-keyed generator):
// with b2 near 1 a step changes sqrt(v) by far less than half a code step, so rounding to nearest
// would never let it decay; in expectation stochastic rounding keeps every change. A root above zero
// never becomes zero: it would be a denominator of eps alone at the next step. A value whose m or v
// is not finite keeps NaN in both, and its block the scales that it would have without it.
// The update itself uses m and v before they are rounded.
//
// Bound by HBM traffic (fp32 states: 26 bytes a value read and written plus the gradient; 8 bits:
// 14.1 plus the gradient). A thread takes 8 consecutive values (16-byte accesses, one generator call
// per state) and 4 lanes share a block of 32; a workgroup takes one chunk of CHUNK values of one
// tensor, found through a table on the device, so any number of tensors is one launch.
#include <math.h>

#include "pmn_dev.hpp"
#include "pmn_kernels.hpp"

namespace pmn {

namespace adw {
constexpr int THREADS = 256;
constexpr int CHUNK = THREADS * 8;   // values per workgroup (chunks of 4 and 8 times as many: 4% and 9% slower)
}  // namespace adw

int64_t adamw_chunk() { return adw::CHUNK; }

// Maximum over the 4 lanes of a quad, in every lane.
PMN_DEV float quad_max4(float v)
{
    v = fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0xB1, 0xF, 0xF, true)));
    return fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x4E, 0xF, 0xF, true)));
}

// n valid values (1..8) of 8 at p
template <typename T>
PMN_DEV void load_values(const T* p, int n, float (&v)[8])
{
    if constexpr (sizeof(T) == 4) {
        if (n == 8) {
            const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
            v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
            v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
            return;
        }
#pragma unroll
        for (int j = 0; j < 8; j++) v[j] = j < n ? (float)p[j] : 0.0f;
    } else {
        if (n == 8) {
            const uint4 w = *reinterpret_cast<const uint4*>(p);
            const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int q = 0; q < 4; q++) {
                v[2 * q] = bf16_lo(a[q]);
                v[2 * q + 1] = bf16_hi(a[q]);
            }
            return;
        }
#pragma unroll
        for (int j = 0; j < 8; j++) v[j] = j < n ? bf16_lo(p[j]) : 0.0f;
    }
}

PMN_DEV void store_f32(float* p, int n, const float (&v)[8])
{
    if (n == 8) {
        reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; j++)
        if (j < n) p[j] = v[j];
}

PMN_DEV void store_bf16(uint16_t* p, int n, const float (&v)[8])
{
    const uint32_t w[4] = {bf16x2_bits(v[0], v[1]), bf16x2_bits(v[2], v[3]), bf16x2_bits(v[4], v[5]),
                           bf16x2_bits(v[6], v[7])};
    if (n == 8) {
        *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; j++)
        if (j < n) p[j] = (uint16_t)(j & 1 ? w[j >> 1] >> 16 : w[j >> 1]);
}

// 8 codes (bytes of n values) and their block's scale -> fp32
PMN_DEV void load_codes(const uint8_t* p, int n, float scale, float (&v)[8])
{
    uint32_t w[2] = {0u, 0u};
    if (n == 8) {
        const uint2 a = *reinterpret_cast<const uint2*>(p);
        w[0] = a.x;
        w[1] = a.y;
    } else {
#pragma unroll
        for (int j = 0; j < 8; j++)
            if (j < n) w[j >> 2] |= (uint32_t)p[j] << (8 * (j & 3));
    }
#pragma unroll
    for (int q = 0; q < 2; q++) {
        const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[q], false);
        const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[q], true);
        v[4 * q] = lo.x * scale;
        v[4 * q + 1] = lo.y * scale;
        v[4 * q + 2] = hi.x * scale;
        v[4 * q + 3] = hi.y * scale;
    }
}

// Lane L of each quad, in every lane of it
template <int L>
PMN_DEV float quad_lane(float v)
{
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x55 * L, 0xF, 0xF, true));
}

// Largest magnitude of a block held by the 4 lanes of a quad, NaN left out
PMN_DEV float block_max(const float (&v)[8])
{
    float amax = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; j++) amax = fmaxf(amax, fabsf(v[j]));
    return quad_max4(amax);
}

// 2^-e as torch.ldexp forms it, by powf, so that states packed by torch operations have the same codes.
// powf is one ulp low for some e, where one of 65536 values on the grid gets the code below it; it is
// held to 2^-e, for one ulp high would put a block's largest value past 448. (The exact power: 460 us for
// 150 M values against 464.)
PMN_DEV float block_scale(int e) { return fminf(powf(2.0f, (float)-e), __builtin_ldexpf(1.0f, -e)); }

// 8 values of a block of exponent e: stochastic E4M3 codes of v * scale; the quad's first lane writes
// the E8M0 byte. POSITIVE: values >= 0, one above zero gets at least the smallest code.
template <bool POSITIVE>
PMN_DEV void store_codes(uint8_t* p, uint8_t* e8m0, int n, const float (&v)[8], int e, float scale, uint64_t seed,
                         uint32_t stream, uint64_t blk)
{
    uint32_t rw[4], w[2] = {0u, 0u};
    rand16x8(seed, stream, blk, rw);
#pragma unroll
    for (int j = 0; j < 8; j++) {
        uint32_t c = e4m3_sr(v[j] * scale, sr_operand(rw[j >> 1], j & 1));
        if (POSITIVE && v[j] > 0.0f && c == 0u) c = 1u;
        w[j >> 2] |= c << (8 * (j & 3));
    }
    if (n == 8) {
        *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
        for (int j = 0; j < 8; j++)
            if (j < n) p[j] = (uint8_t)(w[j >> 2] >> (8 * (j & 3)));
    }
    if ((threadIdx.x & 3) == 0) *e8m0 = (uint8_t)(e + 127);
}

// 1 / (1 - beta1^t) and 1 / sqrt(1 - beta2^t): in fp64 on the host, or here for a step on the device
PMN_DEV void bias_corrections(const AdamwScalars& a, int64_t step, float& ibc1, float& rsbc2)
{
    ibc1 = (float)(-1.0 / expm1((double)step * a.ln_beta1));
    rsbc2 = (float)(1.0 / sqrt(-expm1((double)step * a.ln_beta2)));
}

template <bool EIGHT>
__global__ __launch_bounds__(adw::THREADS) void k_adamw(const AdamwTable* __restrict__ table, AdamwScalars a)
{
    // a table of other states or of fewer chunks than the caller says is not run
    if (table->magic != ADAMW_MAGIC || table->bits != (EIGHT ? 8 : 32) || (int64_t)blockIdx.x >= table->chunks) return;
    const AdamwEntry* entries = reinterpret_cast<const AdamwEntry*>(table + 1);
    const AdamwChunk* map = reinterpret_cast<const AdamwChunk*>(entries + table->count);
    const AdamwChunk ck = map[blockIdx.x];
    const AdamwEntry t = entries[ck.tensor];

    int64_t step = a.step;
    const float lr = a.lr_dev ? *a.lr_dev : a.lr;
    const float gs = a.grad_scale_dev ? *a.grad_scale_dev : 1.0f;
    float ibc1 = a.ibc1, rsbc2 = a.rsbc2;
    if (a.step_dev) {
        step = *a.step_dev;
        step = step < 1 ? 1 : step;
        bias_corrections(a, step, ibc1, rsbc2);
    }
    const float decay = 1.0f - lr * t.weight_decay;
    const float lrm = lr * ibc1;

    const int64_t i0 = (int64_t)ck.index * adw::CHUNK + threadIdx.x * 8;
    // lanes past the tensor's end take no part in its loads and stores, but their quad's amax may
    // need them as zeros: a quad is left only as a whole
    if ((i0 & ~(int64_t)31) >= t.n) return;
    const int64_t left = t.n - i0;
    const int n = left >= 8 ? 8 : (left > 0 ? (int)left : 0);

    float p[8], g[8], m[8], v[8];
    load_values(static_cast<const float*>(t.param) + i0, n, p);
    if (t.grad_f32) load_values(static_cast<const float*>(t.grad) + i0, n, g);
    else load_values(static_cast<const uint16_t*>(t.grad) + i0, n, g);
    if constexpr (EIGHT) {
        const float ms = __builtin_ldexpf(1.0f, (int)t.m_e8m0[i0 >> 5] - 127);
        const float vs = __builtin_ldexpf(1.0f, (int)t.v_e8m0[i0 >> 5] - 127);
        load_codes(static_cast<const uint8_t*>(t.m) + i0, n, ms, m);
        load_codes(static_cast<const uint8_t*>(t.v) + i0, n, vs, v);
#pragma unroll
        for (int j = 0; j < 8; j++) v[j] = v[j] * v[j];
    } else {
        load_values(static_cast<const float*>(t.m) + i0, n, m);
        load_values(static_cast<const float*>(t.v) + i0, n, v);
    }
    float root[8];
#pragma unroll
    for (int j = 0; j < 8; j++) {
        const float gj = g[j] * gs;
        // each product and sum rounded by itself (no fma): the moments' bits, and with them the
        // choices of the stochastic rounding, are those of the formula as written
        m[j] = a.beta1 * m[j] + a.one_minus_beta1 * gj;
        v[j] = a.beta2 * v[j] + a.one_minus_beta2 * gj * gj;
        root[j] = sqrtf(v[j]);
        const float d = __builtin_fmaf(root[j], rsbc2, a.eps);
        p[j] = __builtin_fmaf(-lrm, m[j] / d, p[j] * decay);
    }
    if (n > 0) {
        store_f32(static_cast<float*>(t.param) + i0, n, p);
        if (t.copy) store_bf16(static_cast<uint16_t*>(t.copy) + i0, n, p);
    }
    if constexpr (EIGHT) {
        const uint64_t seed = a.seed + (uint64_t)step, blk = (uint64_t)i0 >> 3;
        const uint32_t stream = a.rng_stream + 2u * (uint32_t)ck.tensor;
        // An infinity would be its block's scale, and the 31 other values' moments zeros and roots too large
        // to square: where one is (the same in all lanes of a quad), a value whose m or v is not finite gets
        // NaN for both, which no scale counts.
        float am = block_max(m), ar = block_max(root);
        if (fmaxf(am, ar) == INFINITY) {
#pragma unroll
            for (int j = 0; j < 8; j++)
                if (!(fabsf(m[j]) < INFINITY && root[j] < INFINITY)) m[j] = root[j] = NAN;
            am = block_max(m);
            ar = block_max(root);
        }
        const int em = e8m0_exponent<E8M0_E4M3>(am), ev = e8m0_exponent<E8M0_E4M3>(ar);
        // both scales, one powf a lane: even lanes of a quad take m's, odd ones v's
        const float inv = block_scale(threadIdx.x & 1 ? ev : em);
        store_codes<false>(static_cast<uint8_t*>(t.m) + i0, t.m_e8m0 + (i0 >> 5), n, m, em, quad_lane<0>(inv), seed,
                           stream, blk);
        store_codes<true>(static_cast<uint8_t*>(t.v) + i0, t.v_e8m0 + (i0 >> 5), n, root, ev, quad_lane<1>(inv), seed,
                          stream + 1u, blk);
    } else if (n > 0) {
        store_f32(static_cast<float*>(t.m) + i0, n, m);
        store_f32(static_cast<float*>(t.v) + i0, n, v);
    }
}

hipError_t launch_adamw(const void* table, int64_t chunks, int bits, const AdamwScalars& a, hipStream_t stream)
{
    const AdamwTable* t = static_cast<const AdamwTable*>(table);
    if (bits == 8)
        hipLaunchKernelGGL((k_adamw<true>), dim3((unsigned)chunks), dim3(adw::THREADS), 0, stream, t, a);
    else
        hipLaunchKernelGGL((k_adamw<false>), dim3((unsigned)chunks), dim3(adw::THREADS), 0, stream, t, a);
    return hipGetLastError();
}

}  // namespace pmn
