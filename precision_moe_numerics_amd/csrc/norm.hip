// norm.hip -- root-mean-square norm with the residual's addition, before the expert layer, with
// its output in bf16 and / or MXFP8, and its backward.
//
// Forward, per row of C values:
//     z = x + r,   s = 1 / sqrt(mean(z^2) + eps),   y = z s gamma
// z (the residual stream after the addition) is written in r's type; the norm uses the sum itself, so
// y is rounded once. MXFP8 codes take y itself, not the bf16 output: e is the smallest exponent with
// max|y| <= 448 * 2^e over 32 values, code = E4M3(y 2^-e) to nearest even.
// Backward, with xh = z s and t = dy gamma:
//     dz = s (t - xh mean(t xh)) + dres,   dgamma = sum over rows of dy xh
//
// Both are bound by HBM traffic: every value is read once into registers (a row is held by one
// wavefront, 512 or 1024 threads, in 16-byte pieces of 8 values) and written once: 16384 rows of 4096
// with a bf16 residual move 606 MB forward (y and codes out) in 104 us, 537 MB backward in 104 us, 5.8
// and 5.2 TB/s where a copy of 1 GB reaches 5.1. Sums (fp64 forward, fp32 backward) take a thread's
// values in order, then a butterfly over the lanes, then the wavefronts in order, so results do not
// depend on the launch.
#include "pmn_dev.hpp"
#include "pmn_kernels.hpp"

namespace pmn {

template <typename S>
PMN_DEV S wave_sum(S v)
{
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m, 64);
    return v;
}

// Maximum over the 4 lanes of a quad (the 32 values of one MXFP8 block), in every lane.
PMN_DEV float quad_max(float v)
{
    v = fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0xB1, 0xF, 0xF, true)));
    return fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x4E, 0xF, 0xF, true)));
}

// 8 consecutive values as fp32, and back (bf16: round to nearest even)
PMN_DEV void load8(const uint16_t* p, float (&v)[8])
{
    const uint4 w = *reinterpret_cast<const uint4*>(p);
    const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int q = 0; q < 4; q++) {
        v[2 * q] = bf16_lo(a[q]);
        v[2 * q + 1] = bf16_hi(a[q]);
    }
}
PMN_DEV void load8(const float* p, float (&v)[8])
{
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
PMN_DEV void store8(uint16_t* p, const float (&v)[8])
{
    *reinterpret_cast<uint4*>(p) = make_uint4(bf16x2_bits(v[0], v[1]), bf16x2_bits(v[2], v[3]),
                                              bf16x2_bits(v[4], v[5]), bf16x2_bits(v[6], v[7]));
}
PMN_DEV void store8(float* p, const float (&v)[8])
{
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// Sum over the T threads of a row. red: T / 64 values (two sets used in turn by a loop over rows,
// so one barrier per row is enough). T = 64: the wavefront alone.
template <int T, typename S>
PMN_DEV S row_sum(S v, S* red)
{
    v = wave_sum(v);
    if (T == 64) return v;
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    S s = 0;
#pragma unroll
    for (int w = 0; w < T / 64; w++) s += red[w];
    return s;
}

// One row per T threads, CH pieces of 8 values each. R: the residual's type (uint8_t: none).
template <int T, int CH, typename R>
__global__ __launch_bounds__(T < 256 ? 256 : T) void k_rmsnorm_fwd(
    const uint16_t* __restrict__ x, const R* res, const float* __restrict__ gamma, float eps,
    int64_t rows, int C, R* z_out, uint16_t* __restrict__ y, uint8_t* __restrict__ codes,
    uint8_t* __restrict__ e8m0, float* __restrict__ rstd)
{
    constexpr bool HAS_RES = !__is_same(R, uint8_t);
    constexpr int RPB = T < 256 ? 256 / T : 1;
    __shared__ double red[T / 64];
    const int t = threadIdx.x % T;
    const int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / T;
    if (row >= rows) return;   // whole wavefronts (T >= 64); with T > 64 the whole workgroup
    const int nch = C >> 3;
    // An error of y turns the E4M3 codes that lie next to a tie: the squares are summed in fp64, and the
    // errors of s and of the products (from fma) are put back before the codes. (y in fp64, or with z's
    // own rounding and the last one put back too, turned no code and was 4 to 10% slower.)
    float z[CH][8];
    double ss = 0.0;
#pragma unroll
    for (int i = 0; i < CH; i++) {
        const int c = t + i * T;
        if (c < nch) {
            load8(x + row * C + 8 * c, z[i]);
            if constexpr (HAS_RES) {
                float r[8];
                load8(res + row * C + 8 * c, r);
#pragma unroll
                for (int j = 0; j < 8; j++) z[i][j] += r[j];
                store8(z_out + row * C + 8 * c, z[i]);
            }
#pragma unroll
            for (int j = 0; j < 8; j++) ss = __builtin_fma((double)z[i][j], (double)z[i][j], ss);
        }
    }
    ss = row_sum<T>(ss, red);
    const double sd = 1.0 / sqrt(ss / (double)C + (double)eps);
    const float s = (float)sd, sl = (float)(sd - (double)s);
    if (rstd && t == 0) rstd[row] = s;
#pragma unroll
    for (int i = 0; i < CH; i++) {
        const int c = t + i * T;
        if (c < nch) {
            float g[8];
            load8(gamma + 8 * c, g);
#pragma unroll
            for (int j = 0; j < 8; j++) {
                const float v = z[i][j], p = v * s, e = __builtin_fmaf(v, sl, __builtin_fmaf(v, s, -p));
                z[i][j] = __builtin_fmaf(p, g[j], e * g[j]);
            }
            if (y) store8(y + row * C + 8 * c, z[i]);
            if (codes) {
                float amax = 0.0f;
#pragma unroll
                for (int j = 0; j < 8; j++) amax = fmaxf(amax, fabsf(z[i][j]));
                const int e = e8m0_exponent<E8M0_E4M3>(quad_max(amax));
                float q[8];
#pragma unroll
                for (int j = 0; j < 8; j++) q[j] = __builtin_ldexpf(z[i][j], -e);
                int lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
                lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], lo, true);
                int hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[4], q[5], 0, false);
                hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[6], q[7], hi, true);
                *reinterpret_cast<uint2*>(codes + row * C + 8 * c) = make_uint2((uint32_t)lo, (uint32_t)hi);
                if ((t & 3) == 0) e8m0[row * (C >> 5) + (c >> 2)] = (uint8_t)(e + 127);
            }
        }
    }
}

// Rows row0, row0 + stride, ... of one T-thread group; dgamma sums stay in registers and leave as
// one partial row per workgroup.
template <int T, int CH, typename Z, typename D>
__global__ __launch_bounds__(T < 256 ? 256 : T) void k_rmsnorm_bwd(
    const D* __restrict__ dy, const Z* __restrict__ zin, const float* __restrict__ gamma,
    const float* __restrict__ rstd, const Z* dres, int64_t rows, int C, Z* dz,
    float* __restrict__ part)
{
    constexpr int RPB = T < 256 ? 256 / T : 1;
    __shared__ float red[2][T / 64];
    __shared__ float comb[RPB > 1 ? RPB - 1 : 1][RPB > 1 ? T * CH * 8 : 1];
    const int t = threadIdx.x % T, grp = threadIdx.x / T;
    const int nch = C >> 3;
    const float invC = 1.0f / (float)C;
    float dg[CH][8];
#pragma unroll
    for (int i = 0; i < CH; i++)
#pragma unroll
        for (int j = 0; j < 8; j++) dg[i][j] = 0.0f;
    int k = 0;
    for (int64_t row = (int64_t)blockIdx.x * RPB + grp; row < rows; row += (int64_t)gridDim.x * RPB, k ^= 1) {
        const float s = rstd[row];
        float xh[CH][8], tt[CH][8];
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < CH; i++) {
            const int c = t + i * T;
            if (c < nch) {
                float g[8];
                load8(zin + row * C + 8 * c, xh[i]);
                load8(dy + row * C + 8 * c, tt[i]);
                load8(gamma + 8 * c, g);
#pragma unroll
                for (int j = 0; j < 8; j++) {
                    xh[i][j] *= s;
                    dg[i][j] = __builtin_fmaf(tt[i][j], xh[i][j], dg[i][j]);
                    tt[i][j] *= g[j];
                    dot = __builtin_fmaf(tt[i][j], xh[i][j], dot);
                }
            }
        }
        dot = row_sum<T>(dot, red[k]) * invC;
#pragma unroll
        for (int i = 0; i < CH; i++) {
            const int c = t + i * T;
            if (c < nch) {
                float r[8];
                if (dres) {
                    load8(dres + row * C + 8 * c, r);
                } else {
#pragma unroll
                    for (int j = 0; j < 8; j++) r[j] = 0.0f;
                }
#pragma unroll
                for (int j = 0; j < 8; j++)
                    tt[i][j] = __builtin_fmaf(s, __builtin_fmaf(-xh[i][j], dot, tt[i][j]), r[j]);
                store8(dz + row * C + 8 * c, tt[i]);
            }
        }
    }
    if constexpr (RPB > 1) {
        if (grp > 0) {
#pragma unroll
            for (int i = 0; i < CH; i++)
#pragma unroll
                for (int j = 0; j < 8; j++) comb[grp - 1][(i * T + t) * 8 + j] = dg[i][j];
        }
        __syncthreads();
        if (grp == 0) {
#pragma unroll
            for (int i = 0; i < CH; i++)
#pragma unroll
                for (int w = 0; w < RPB - 1; w++)
#pragma unroll
                    for (int j = 0; j < 8; j++) dg[i][j] += comb[w][(i * T + t) * 8 + j];
        }
    }
    if (grp == 0) {
#pragma unroll
        for (int i = 0; i < CH; i++) {
            const int c = t + i * T;
            if (c < nch) store8(part + (int64_t)blockIdx.x * C + 8 * c, dg[i]);
        }
    }
}

// dgamma[c] = sum of the P partial rows: 32 columns a workgroup (a 128-byte line of each row), 32
// threads down the rows of each column, their sums added in order.
__global__ __launch_bounds__(1024) void k_rmsnorm_dgamma(const float* __restrict__ part, int P, int C,
                                                         float* __restrict__ dgamma)
{
    __shared__ float red[32][33];
    const int x = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + x;
    float s = 0.0f;
    if (c < C) {
#pragma unroll 8
        for (int p = w; p < P; p += 32) s += part[(int64_t)p * C + c];
    }
    red[w][x] = s;
    __syncthreads();
    if (w == 0 && c < C) {
#pragma unroll
        for (int i = 1; i < 32; i++) s += red[i][x];
        dgamma[c] = s;
    }
}

__global__ void k_zero_f32(float* __restrict__ p, int64_t n)
{
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i < n) p[i] = 0.0f;
}

// Threads per row and pieces per thread: rows of up to 2048 values go to one wavefront (no barrier),
// longer ones to as many threads as pieces up to 1024, so that a row's latency is shared by more
// wavefronts (against 256 threads: 8000 rows of 7168 forward 100 -> 91 us, backward 117 -> 77 us;
// 16384 rows of 4096 forward 110.5 -> 107 us, backward the same).
#define PMN_NORM_DISPATCH(C)                              \
    do {                                                  \
        const int nch_ = (int)((C) >> 3);                 \
        if (nch_ <= 64) { PMN_CALL(64, 1); }              \
        else if (nch_ <= 128) { PMN_CALL(64, 2); }        \
        else if (nch_ <= 256) { PMN_CALL(64, 4); }        \
        else if (nch_ <= 512) { PMN_CALL(512, 1); }       \
        else if (nch_ <= 1024) { PMN_CALL(1024, 1); }     \
        else if (nch_ <= 2048) { PMN_CALL(1024, 2); }     \
        else { PMN_CALL(1024, 4); }                       \
    } while (0)

template <typename R>
static void rmsnorm_fwd_typed(const uint16_t* x, const R* res, const float* gamma, float eps, int64_t rows, int64_t C,
                              R* z, uint16_t* y, uint8_t* codes, uint8_t* e8m0, float* rstd, hipStream_t stream)
{
    // a launch holds fewer than 2^32 threads: at most 2^31 / T rows in one
#define PMN_CALL(T, CH)                                                                                            \
    for (int64_t r0 = 0; r0 < rows; r0 += ((int64_t)1 << 31) / (T)) {                                              \
        const int64_t most = ((int64_t)1 << 31) / (T), n = rows - r0 < most ? rows - r0 : most, o = r0 * C;        \
        const int rpb = (T) < 256 ? 256 / (T) : 1;                                                                 \
        hipLaunchKernelGGL((k_rmsnorm_fwd<T, CH, R>), dim3((unsigned)((n + rpb - 1) / rpb)),                       \
                           dim3((T) < 256 ? 256 : (T)), 0, stream, x + o, res ? res + o : nullptr, gamma, eps, n,  \
                           (int)C, z ? z + o : nullptr, y ? y + o : nullptr, codes ? codes + o : nullptr,          \
                           e8m0 ? e8m0 + o / 32 : nullptr, rstd ? rstd + r0 : nullptr);                            \
    }
    PMN_NORM_DISPATCH(C);
#undef PMN_CALL
}

hipError_t launch_rmsnorm_fwd(const uint16_t* x, const void* res, bool res_f32, const float* gamma, float eps,
                              int64_t rows, int64_t C, void* z, uint16_t* y, uint8_t* codes, uint8_t* e8m0,
                              float* rstd, hipStream_t stream)
{
    if (!res) {
        rmsnorm_fwd_typed<uint8_t>(x, nullptr, gamma, eps, rows, C, nullptr, y, codes, e8m0, rstd, stream);
    } else if (res_f32) {
        rmsnorm_fwd_typed<float>(x, static_cast<const float*>(res), gamma, eps, rows, C, static_cast<float*>(z), y,
                                 codes, e8m0, rstd, stream);
    } else {
        rmsnorm_fwd_typed<uint16_t>(x, static_cast<const uint16_t*>(res), gamma, eps, rows, C,
                                    static_cast<uint16_t*>(z), y, codes, e8m0, rstd, stream);
    }
    return hipGetLastError();
}

// Workgroups of the backward = partial rows of dgamma: enough to fill the chip, few enough that the
// partials stay small beside the rows (at 1024 they are half of the traffic of 1000 rows: 7168 values
// wide 22 us, at 512 15). Rows over 1024 threads fill half of a CU each: up to 1024 of them go to 256
// workgroups, which halves the partials. 512 against 256 workgroups, us (rows of 4104 to 32768 values,
// 300 to 1024 of them, in either type: never more than 2% slower with 256):
//     bf16  640 x 4608 12.0, 11.8   640 x 7168 14.0, 12.7   1024 x 12288 27.0, 23.5   1024 x 32768 83.7, 71.4
//     fp32  640 x 4608 13.7, 13.1   640 x 7168 19.9, 17.4   1024 x 12288 42.8, 36.5   1024 x 32768 157, 142
// 2500 rows go the other way up to 8192 values (bf16 of 4608 19.7, 21.7), and so do shorter rows (fp32 of
// 4096 over 512 threads: 777 rows 14.4, 14.7). A function of the sizes alone, so results are too.
static int64_t rmsnorm_bwd_groups(int64_t rows, int64_t C)
{
    const int64_t rpb = C <= 2048 ? 4 : 1;
    const int64_t n = (rows + rpb - 1) / rpb;
    const int64_t most = C > 4096 && rows <= 1024 ? 256 : 512;
    return n < most ? n : most;
}

size_t rmsnorm_bwd_ws_bytes(int64_t rows, int64_t C)
{
    return (size_t)rmsnorm_bwd_groups(rows, C) * (size_t)C * sizeof(float);
}

template <typename Z, typename D>
static void rmsnorm_bwd_typed(const D* dy, const Z* z, const float* gamma, const float* rstd, const Z* dres,
                              int64_t rows, int64_t C, Z* dz, float* part, hipStream_t stream)
{
    const unsigned grid = (unsigned)rmsnorm_bwd_groups(rows, C);
#define PMN_CALL(T, CH)                                                                                         \
    hipLaunchKernelGGL((k_rmsnorm_bwd<T, CH, Z, D>), dim3(grid), dim3((T) < 256 ? 256 : (T)), 0, stream, dy, z, \
                       gamma, rstd, dres, rows, (int)C, dz, part)
    PMN_NORM_DISPATCH(C);
#undef PMN_CALL
}

hipError_t launch_rmsnorm_bwd(const void* dy, bool dy_f32, const void* z, bool z_f32, const float* gamma,
                              const float* rstd, const void* dres, int64_t rows, int64_t C, void* dz, float* dgamma,
                              float* part, hipStream_t stream)
{
    if (rows == 0) {
        hipLaunchKernelGGL(k_zero_f32, dim3((unsigned)((C + 255) / 256)), dim3(256), 0, stream, dgamma, C);
        return hipGetLastError();
    }
#define PMN_TYPED(Z, D)                                                                                            \
    rmsnorm_bwd_typed<Z, D>(static_cast<const D*>(dy), static_cast<const Z*>(z), gamma, rstd,                      \
                            static_cast<const Z*>(dres), rows, C, static_cast<Z*>(dz), part, stream)
    if (z_f32 && dy_f32) PMN_TYPED(float, float);
    else if (z_f32) PMN_TYPED(float, uint16_t);
    else if (dy_f32) PMN_TYPED(uint16_t, float);
    else PMN_TYPED(uint16_t, uint16_t);
#undef PMN_TYPED
    hipLaunchKernelGGL(k_rmsnorm_dgamma, dim3((unsigned)((C + 31) / 32)), dim3(1024), 0, stream, part,
                       (int)rmsnorm_bwd_groups(rows, C), (int)C, dgamma);
    return hipGetLastError();
}

}  // namespace pmn
