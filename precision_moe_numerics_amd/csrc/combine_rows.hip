// combine_rows.hip -- the experts' unquantized rows back to their tokens, and the gradient:
//     out[t] = sum_j gates[t, j] y[slot_of[t, j]] (+ add[t])
//     dy[slot_of[t, j]] = gates[t, j] dout[t],   dgates[t, j] = <dout[t], y[slot_of[t, j]]>
// Both are bound by HBM: each row of y is read once (and of dy written once), a token's row once. Sums are
// fp32 in the order of j (dgates: a fixed tree), outputs rounded once.
//
// Forward: a thread holds 8 consecutive values of a token's row and has up to 8 slots' words on the way.
// Backward: a workgroup takes a token, holds each word of dout for 8 slots at a time and sums their dot
// products side by side, so that their wavefronts' sums are joined once. Rows of a new dy that no pair names
// get zeros from a launch of their own, which reads slot_of and writes those rows alone.
#include "pmn_dev.hpp"
#include "pmn_kernels.hpp"

namespace pmn {

namespace rows {
constexpr int KB = 8;   // slots at a time

template <bool F32>
struct Words {
    uint4 w[F32 ? 2 : 1];
};

template <bool F32>
PMN_DEV Words<F32> load8(const void* p, int64_t at)
{
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    Words<F32> r;
    const u32x4* q = reinterpret_cast<const u32x4*>(static_cast<const uint8_t*>(p) + at * (F32 ? 4 : 2));
#pragma unroll
    for (int i = 0; i < (F32 ? 2 : 1); i++) {
        const u32x4 v = __builtin_nontemporal_load(q + i);
        r.w[i] = make_uint4(v.x, v.y, v.z, v.w);
    }
    return r;
}

template <bool F32>
PMN_DEV void values8(const Words<F32>& r, float (&o)[8])
{
    if (F32) {
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const uint4 w = r.w[F32 ? i : 0];
            o[4 * i] = __uint_as_float(w.x);
            o[4 * i + 1] = __uint_as_float(w.y);
            o[4 * i + 2] = __uint_as_float(w.z);
            o[4 * i + 3] = __uint_as_float(w.w);
        }
    } else {
        const uint32_t a[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
        for (int i = 0; i < 4; i++) {
            o[2 * i] = bf16_lo(a[i]);
            o[2 * i + 1] = bf16_hi(a[i]);
        }
    }
}

template <bool F32>
PMN_DEV void store8(void* p, int64_t at, const float (&o)[8])
{
    if (F32) {
        float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + at);
        q[0] = make_float4(o[0], o[1], o[2], o[3]);
        q[1] = make_float4(o[4], o[5], o[6], o[7]);
    } else {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + at) =
            make_uint4(bf16x2_bits(o[0], o[1]), bf16x2_bits(o[2], o[3]), bf16x2_bits(o[4], o[5]), bf16x2_bits(o[6], o[7]));
    }
}

// Slot of pair q (slot_of null: the pair itself), -1 outside [0, M)
PMN_DEV int64_t slot_at(const int32_t* slot_of, int64_t q, int64_t M)
{
    const int64_t s = slot_of ? (int64_t)slot_of[q] : q;
    return s >= 0 && s < M ? s : -1;
}
}  // namespace rows

template <bool YF32, bool OF32>
__global__ __launch_bounds__(256) void k_combine_rows(const void* __restrict__ y, int64_t M, int64_t H,
                                                      const int32_t* __restrict__ slot_of,
                                                      const float* __restrict__ gates, const int32_t* __restrict__ ids, int G,
                                                      const uint16_t* add, int64_t T, int k, int chunks, void* out)
{
    using namespace rows;
    const int64_t t = blockIdx.x / (unsigned)chunks;
    const int64_t h = ((int64_t)(blockIdx.x - t * chunks) * blockDim.x + threadIdx.x) * 8;
    if (h >= H) return;
    float acc[8];
#pragma unroll
    for (int u = 0; u < 8; u++) acc[u] = 0.0f;
    for (int j0 = 0; j0 < k; j0 += KB) {
        Words<YF32> w[KB];
        float gt[KB];
        bool on[KB];
#pragma unroll
        for (int j = 0; j < KB; j++) {
            const int64_t q = t * k + j0 + j, s = j0 + j < k ? slot_at(slot_of, q, M) : -1;
            on[j] = s >= 0 && (!ids || (uint32_t)ids[q] < (uint32_t)G);
            gt[j] = on[j] && gates ? gates[t * k + j0 + j] : 1.0f;
            if (on[j]) w[j] = load8<YF32>(y, s * H + h);
        }
#pragma unroll
        for (int j = 0; j < KB; j++)
            if (on[j]) {
                float v[8];
                values8<YF32>(w[j], v);
#pragma unroll
                for (int u = 0; u < 8; u++) acc[u] = __builtin_fmaf(gt[j], v[u], acc[u]);
            }
    }
    if (add) {
        float v[8];
        values8<false>(load8<false>(add, t * H + h), v);
#pragma unroll
        for (int u = 0; u < 8; u++) acc[u] += v[u];
    }
    store8<OF32>(out, t * H + h, acc);
}

template <bool DF32, bool YF32>
__global__ __launch_bounds__(256) void k_combine_rows_bwd(const void* __restrict__ dout, const void* __restrict__ y,
                                                          int64_t M, int64_t H, const int32_t* __restrict__ slot_of,
                                                          const float* __restrict__ gates, int64_t T, int k,
                                                          void* __restrict__ dy, float* __restrict__ dgates)
{
    using namespace rows;
    __shared__ float part[4][KB];
    const int64_t t = blockIdx.x;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int j0 = 0; j0 < k; j0 += KB) {
        int64_t s[KB];
        float gt[KB], dot[KB];
#pragma unroll
        for (int j = 0; j < KB; j++) {
            s[j] = j0 + j < k ? slot_at(slot_of, t * k + j0 + j, M) : -1;
            gt[j] = s[j] >= 0 && gates ? gates[t * k + j0 + j] : 1.0f;
            dot[j] = 0.0f;
        }
        for (int64_t h = threadIdx.x * 8; h < H; h += blockDim.x * 8) {
            float d[8];
            values8<DF32>(load8<DF32>(dout, t * H + h), d);
            Words<YF32> w[KB];
            if (dgates) {
#pragma unroll
                for (int j = 0; j < KB; j++)
                    if (s[j] >= 0) w[j] = load8<YF32>(y, s[j] * H + h);
            }
#pragma unroll
            for (int j = 0; j < KB; j++) {
                if (s[j] < 0) continue;
                if (dgates) {
                    float v[8];
                    values8<YF32>(w[j], v);
#pragma unroll
                    for (int u = 0; u < 8; u++) dot[j] = __builtin_fmaf(d[u], v[u], dot[j]);
                }
                if (dy) {
                    float v[8];
#pragma unroll
                    for (int u = 0; u < 8; u++) v[u] = gt[j] * d[u];
                    store8<YF32>(dy, s[j] * H + h, v);
                }
            }
        }
        if (dgates) {
#pragma unroll
            for (int j = 0; j < KB; j++)
#pragma unroll
                for (int m = 32; m >= 1; m >>= 1) dot[j] += __shfl_xor(dot[j], m, 64);
            if (j0 > 0) __syncthreads();
            if (lane == 0) {
#pragma unroll
                for (int j = 0; j < KB; j++) part[wave][j] = dot[j];
            }
            __syncthreads();
            const int j = threadIdx.x;
            if (j < KB && j0 + j < k) {
                float v = 0.0f;
                for (unsigned q = 0; q < blockDim.x / 64; q++) v += part[q][j];
                dgates[t * k + j0 + j] = v;   // a slot outside [0, M): zero
            }
        }
    }
}

// Zeros to the rows of x (`words` 16-byte words each) that no pair names. A workgroup marks which of its `per` rows
// are named as bits in LDS, over all pairs, so that nothing but slot_of is read and no memory is shared. Bound by
// a compare and a branch for each pair, in every workgroup: 131072 pairs 12 us where all rows are named (zeros to
// 1 GB of rows beforehand: 156).
__global__ __launch_bounds__(1024) void k_zero_unnamed(const int32_t* __restrict__ slot_of, int64_t pairs, int64_t M,
                                                       int64_t words, int per, uint4* __restrict__ x)
{
    extern __shared__ uint32_t named[];
    const int64_t r0 = (int64_t)blockIdx.x * per;
    const uint32_t n = (uint32_t)(M - r0 < per ? M - r0 : per);
    const int tid = threadIdx.x, lane = tid & 63;
    for (uint32_t i = tid; i < (n + 31) / 32; i += 1024) named[i] = 0;
    __syncthreads();
    auto mark = [&](int32_t s) {   // M < 2^31: what is negative lies past every row
        const uint32_t d = (uint32_t)s - (uint32_t)r0;
        if (d < n) atomicOr(&named[d >> 5], 1u << (d & 31));
    };
    const int64_t quads = reinterpret_cast<uintptr_t>(slot_of) % 16 == 0 ? pairs >> 2 : 0;
    constexpr int AHEAD = 8;   // loads of a thread on their way
    for (int64_t q0 = tid; q0 < quads; q0 += AHEAD * 1024) {
        int4 s[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; i++) {
            const int64_t q = q0 + i * 1024;
            s[i] = reinterpret_cast<const int4*>(slot_of)[q < quads ? q : q0];
        }
#pragma unroll
        for (int i = 0; i < AHEAD; i++) {
            mark(s[i].x);
            mark(s[i].y);
            mark(s[i].z);
            mark(s[i].w);
        }
    }
    for (int64_t q = 4 * quads + tid; q < pairs; q += 1024) mark(slot_of[q]);
    __syncthreads();
    for (uint32_t r = tid >> 6; r < n; r += 16) {
        if (named[r >> 5] >> (r & 31) & 1u) continue;
        uint4* const row = x + (r0 + r) * words;
        for (int64_t h = lane; h < words; h += 64) row[h] = make_uint4(0u, 0u, 0u, 0u);
    }
}

// Threads for rows of H values, 8 a thread: up to 256
static int row_threads(int64_t H) { return H >= 1024 ? 256 : H >= 512 ? 128 : 64; }

hipError_t launch_combine_rows(const void* y, bool y_f32, int64_t M, int64_t H, const int32_t* slot_of,
                               const float* gates, const int32_t* ids, int G, const uint16_t* add, int64_t T, int k,
                               void* out, bool out_f32, hipStream_t stream)
{
    const int th = row_threads(H), chunks = (int)((H / 8 + th - 1) / th);
    // a launch has fewer than 2^32 threads
    const int64_t most = (((int64_t)1 << 32) - 1) / th / chunks;
    for (int64_t t0 = 0; t0 < T; t0 += most) {
        const int64_t n = T - t0 < most ? T - t0 : most;
        const dim3 grid((unsigned)(n * chunks)), block(th);
        const int32_t* so = slot_of ? slot_of + t0 * k : nullptr;
        const float* gt = gates ? gates + t0 * k : nullptr;
        const int32_t* id = ids ? ids + t0 * k : nullptr;
        const uint16_t* ad = add ? add + t0 * H : nullptr;
        const uint8_t* yy = static_cast<const uint8_t*>(y) + (slot_of ? 0 : t0 * k * H * (y_f32 ? 4 : 2));
        const int64_t m = slot_of ? M : M - t0 * k;
        uint8_t* o = static_cast<uint8_t*>(out) + t0 * H * (out_f32 ? 4 : 2);
#define PMN_ROWS(A, B) hipLaunchKernelGGL((k_combine_rows<A, B>), grid, block, 0, stream, yy, m, H, so, gt, id, G, ad, n, k, chunks, o)
        if (y_f32) {
            if (out_f32) PMN_ROWS(true, true);
            else PMN_ROWS(true, false);
        } else {
            if (out_f32) PMN_ROWS(false, true);
            else PMN_ROWS(false, false);
        }
#undef PMN_ROWS
    }
    return hipGetLastError();
}

// T < 2^24
hipError_t launch_combine_rows_bwd(const void* dout, bool d_f32, const void* y, bool y_f32, int64_t M, int64_t H,
                                   const int32_t* slot_of, const float* gates, int64_t T, int k, void* dy,
                                   float* dgates, hipStream_t stream)
{
    const dim3 grid((unsigned)T), block(row_threads(H));
#define PMN_ROWS(A, B) hipLaunchKernelGGL((k_combine_rows_bwd<A, B>), grid, block, 0, stream, dout, y, M, H, slot_of, gates, T, k, dy, dgates)
    if (d_f32) {
        if (y_f32) PMN_ROWS(true, true);
        else PMN_ROWS(true, false);
    } else {
        if (y_f32) PMN_ROWS(false, true);
        else PMN_ROWS(false, false);
    }
#undef PMN_ROWS
    return hipGetLastError();
}

hipError_t launch_zero_unnamed(const int32_t* slot_of, int64_t pairs, int64_t M, int64_t row_bytes, void* x,
                               hipStream_t stream)
{
    // a workgroup a CU, of 2^18 rows (32 KB of bits) at most
    const int64_t even = (M + 255) / 256, most = (int64_t)1 << 18;
    const int per = (int)((even < most ? even : most) + 31) / 32 * 32;
    hipLaunchKernelGGL(k_zero_unnamed, dim3((unsigned)((M + per - 1) / per)), dim3(1024), per / 8, stream, slot_of, pairs, M,
                       row_bytes / 16, per, static_cast<uint4*>(x));
    return hipGetLastError();
}

}  // namespace pmn
