// gdn_norm.cu -- the root-mean-square norms around a Gated DeltaNet layer (include/gdn_layer.h):
// add_rms_norm_fwd, in front of it (the residual's addition, the norm, bf16 or 8 bits out), and
// gated_rms_norm_fwd, behind it (the norm of each head's output, times silu(z)).
//
// Both read every input once and write every output once; a row stays in registers between the sum
// of squares and its use.  Thread t of a row holds the values 8 t .. 8 t + 7 (16 bytes of bf16), so
// the 128 values of an 8-bit group are 16 neighbouring lanes.
#include "gdn_layer.cuh"

namespace kkt {
namespace {

using namespace ptx;

constexpr int kNormMaxDim = 16384;

struct NormParams {
    const void *x, *r, *z, *w;
    void *y, *r_out;
    float *scales;
    int64_t rows;
    int dim, group;
    float eps;
};

// Eight values of a row from element e on: a vector where the row's length and place allow it, else
// one by one; zeros past the row's end.
template <bool VEC, typename T>
__device__ __forceinline__ void row_load(const T *row, int e, int dim, float (&v)[8]) {
    if constexpr (VEC) {
        if (e < dim) {
            widen8(raw8(row + e), v);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = 0.f;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = e + i < dim ? to_f32(row[e + i]) : 0.f;
    }
}
template <bool VEC, typename T>
__device__ __forceinline__ void row_store(T *row, int e, int dim, const float (&v)[8]) {
    if constexpr (VEC) {
        if (e < dim) store8(row + e, v);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (e + i < dim) row[e + i] = from_f32<T>(v[i]);
    }
}

// Sum or maximum over the block; every thread gets it.  `part` holds one value for each warp.
template <bool MAX>
__device__ __forceinline__ float block_reduce(float v, float *part, int warps) {
    v = MAX ? lanes_max<32>(v) : lanes_sum<32>(v);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    float total = part[0];
    for (int i = 1; i < warps; ++i) total = MAX ? fmaxf(total, part[i]) : total + part[i];
    return total;
}

// One block a row, NV groups of eight values to a thread.
template <typename IO, typename OUT, int NV, bool VEC>
__global__ void __launch_bounds__(NV == 4 ? 512 : 256) add_rms_norm_kernel(const NormParams p) {
    __shared__ float part[2][16];
    griddep_launch_dependents();
    griddep_wait();
    const int64_t at = (int64_t)blockIdx.x * p.dim;
    const int step = blockDim.x * 8, e0 = threadIdx.x * 8;
    float h[NV][8];
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) row_load<VEC>(static_cast<const IO *>(p.x) + at, e0 + j * step, p.dim, h[j]);
    if (p.r) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            float r[8];
            row_load<VEC>(static_cast<const IO *>(p.r) + at, e0 + j * step, p.dim, r);
#pragma unroll
            for (int e = 0; e < 8; ++e) h[j][e] += r[e];
        }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(h[j][e], h[j][e], ss);
        if (p.r_out) row_store<VEC>(static_cast<IO *>(p.r_out) + at, e0 + j * step, p.dim, h[j]);
    }
    const int warps = blockDim.x >> 5;
    const float r = rsqrtf(block_reduce<false>(ss, part[0], warps) / (float)p.dim + p.eps);
    float top = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        float w[8];
        row_load<VEC>(static_cast<const IO *>(p.w), e0 + j * step, p.dim, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) h[j][e] *= r * w[e];
        if constexpr (sizeof(OUT) == 1) {
            float m = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(h[j][e]));
            if (p.group) {
                float inv;
                const float s = e4m3_scale(lanes_max<16>(m), inv);
                const int e = e0 + j * step;
                if ((threadIdx.x & 15) == 0 && e < p.dim)
                    p.scales[(int64_t)blockIdx.x * ((p.dim + 127) / 128) + e / 128] = s;
#pragma unroll
                for (int i = 0; i < 8; ++i) h[j][i] *= inv;
            } else {
                top = fmaxf(top, m);
            }
        }
    }
    if constexpr (sizeof(OUT) == 1) {
        if (!p.group) {
            float inv;
            const float s = e4m3_scale(block_reduce<true>(top, part[1], warps), inv);
            if (threadIdx.x == 0) p.scales[blockIdx.x] = s;
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int e = 0; e < 8; ++e) h[j][e] *= inv;
        }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) row_store<VEC>(static_cast<OUT *>(p.y) + at, e0 + j * step, p.dim, h[j]);
}

// DIM / 8 lanes a row, kGatedRows rows to a thread, whose loads are in flight together.
constexpr int kGatedRows = 4;
template <typename IO, typename OUT, int DIM>
__global__ void __launch_bounds__(256) gated_rms_norm_kernel(const NormParams p) {
    constexpr int L = DIM / 8, PER = 256 / L;  // lanes of a row; rows of the block at a time
    griddep_launch_dependents();
    griddep_wait();
    const int e = (threadIdx.x % L) * 8;
    const int64_t row0 = (int64_t)blockIdx.x * (PER * kGatedRows) + threadIdx.x / L;
    const int left = (int)(p.rows - row0 < PER * kGatedRows ? p.rows - row0 : PER * kGatedRows);  // may be negative
    float2 w[4];
    widen8(raw8(static_cast<const IO *>(p.w) + e), w);
    const IO *px = static_cast<const IO *>(p.x) + row0 * DIM + e, *pz = static_cast<const IO *>(p.z) + row0 * DIM + e;
    Raw8<IO> xr[kGatedRows] = {}, zr[kGatedRows] = {};
#pragma unroll
    for (int i = 0; i < kGatedRows; ++i)
        if (i * PER < left) {
            xr[i] = raw8(px + i * PER * DIM);
            zr[i] = raw8(pz + i * PER * DIM);
        }
#pragma unroll
    for (int i = 0; i < kGatedRows; ++i) {
        const bool live = i * PER < left;
        float2 x[4], z[4];
        widen8(xr[i], x);
        widen8(zr[i], z);
        float2 ss = mul2(x[0], x[0]);
#pragma unroll
        for (int j = 1; j < 4; ++j) ss = fma2(x[j], x[j], ss);
        const float r = rsqrtf(lanes_sum<L>(ss.x + ss.y) * (1.f / DIM) + p.eps);
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = mul2(mul2(mul2(x[j], make_float2(r, r)), w[j]), silu2(z[j]));
        if constexpr (sizeof(OUT) == 1) {
            float m = 0.f, inv;
#pragma unroll
            for (int j = 0; j < 4; ++j) m = fmaxf(m, fmaxf(fabsf(x[j].x), fabsf(x[j].y)));
            const float s = e4m3_scale(lanes_max<L>(m), inv);
            if (e == 0 && live) p.scales[row0 + i * PER] = s;
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = mul2(x[j], make_float2(inv, inv));
        }
        if (live) store8(static_cast<OUT *>(p.y) + row0 * DIM + e + i * PER * DIM, x);
    }
}

template <typename IO, typename OUT, int NV>
int launch_add(const NormParams &p, int threads, bool vec, cudaStream_t st) {
    const dim3 grid((unsigned)p.rows);
    return vec ? launch_serialised(add_rms_norm_kernel<IO, OUT, NV, true>, grid, threads, 0, st, p)
               : launch_serialised(add_rms_norm_kernel<IO, OUT, NV, false>, grid, threads, 0, st, p);
}

template <typename IO, typename OUT>
int launch_add(const NormParams &p, bool vec, cudaStream_t st) {
    const int groups = (p.dim + 7) / 8;  // threads that one group each would take
    auto threads = [&](int nv) { return ((groups + nv - 1) / nv + 31) / 32 * 32; };
    if (groups <= 256) return launch_add<IO, OUT, 1>(p, threads(1), vec, st);
    if (groups <= 512) return launch_add<IO, OUT, 2>(p, threads(2), vec, st);
    return launch_add<IO, OUT, 4>(p, threads(4), vec, st);
}

template <typename IO>
int launch_add(const NormParams &p, int out, bool vec, cudaStream_t st) {
    switch (out) {
        case GDN_OUT_BF16: return launch_add<IO, __nv_bfloat16>(p, vec, st);
        case GDN_OUT_F32: return launch_add<IO, float>(p, vec, st);
        default: return launch_add<IO, __nv_fp8_e4m3>(p, vec, st);
    }
}

template <typename IO, typename OUT>
int launch_gated(const NormParams &p, cudaStream_t st) {
    const int64_t per = (int64_t)256 / (p.dim / 8) * kGatedRows;
    const dim3 grid((unsigned)((p.rows + per - 1) / per));
    return p.dim == 128 ? launch_serialised(gated_rms_norm_kernel<IO, OUT, 128>, grid, 256, 0, st, p)
                        : launch_serialised(gated_rms_norm_kernel<IO, OUT, 64>, grid, 256, 0, st, p);
}

template <typename IO>
int launch_gated(const NormParams &p, int out, cudaStream_t st) {
    switch (out) {
        case GDN_OUT_BF16: return launch_gated<IO, __nv_bfloat16>(p, st);
        case GDN_OUT_F32: return launch_gated<IO, float>(p, st);
        default: return launch_gated<IO, __nv_fp8_e4m3>(p, st);
    }
}

bool types_ok(int io, int out) {
    return (io == KKT_IO_BF16 || io == KKT_IO_F32) && out >= GDN_OUT_BF16 && out <= GDN_OUT_E4M3;
}

}  // namespace
}  // namespace kkt

extern "C" int add_rms_norm_fwd(const void *x, const void *residual, const void *weight, int64_t rows, int dim,
                                float eps, int io_dtype, int out_dtype, int group, void *y, float *scales,
                                void *residual_out, struct CUstream_st *stream) {
    using namespace kkt;
    if (rows < 0 || rows > 0x7fffffffLL || dim < 1 || !types_ok(io_dtype, out_dtype)) return KKT_ERR_ARG;
    if (dim > kNormMaxDim) return KKT_ERR_UNSUPPORTED;
    if (group != 0 && group != 128) return KKT_ERR_UNSUPPORTED;
    if (!weight || (rows > 0 && (!x || !y || (out_dtype == GDN_OUT_E4M3 && !scales)))) return KKT_ERR_ARG;
    if (!aligned_ptr(x, 16) || !aligned_ptr(residual, 16) || !aligned_ptr(weight, 16) || !aligned_ptr(y, 16) ||
        !aligned_ptr(residual_out, 16) || !aligned_ptr(scales, 4))
        return KKT_ERR_ALIGN;
    if (rows == 0) return KKT_OK;
    NormParams p;
    p.x = x; p.r = residual; p.z = nullptr; p.w = weight; p.y = y; p.r_out = residual_out; p.scales = scales;
    p.rows = rows; p.dim = dim; p.group = group; p.eps = eps;
    const bool vec = dim % 8 == 0;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return io_dtype == KKT_IO_BF16 ? launch_add<__nv_bfloat16>(p, out_dtype, vec, st)
                                   : launch_add<float>(p, out_dtype, vec, st);
}

extern "C" int gated_rms_norm_fwd(const void *x, const void *z, const void *weight, int64_t rows, int dim, float eps,
                                  int io_dtype, int out_dtype, void *y, float *scales, struct CUstream_st *stream) {
    using namespace kkt;
    if (rows < 0 || dim < 1 || !types_ok(io_dtype, out_dtype)) return KKT_ERR_ARG;
    if (dim != 64 && dim != 128) return KKT_ERR_UNSUPPORTED;
    if (rows / 64 > 0x7ffffff0LL) return KKT_ERR_ARG;
    if (!weight || (rows > 0 && (!x || !z || !y || (out_dtype == GDN_OUT_E4M3 && !scales)))) return KKT_ERR_ARG;
    if (!aligned_ptr(x, 16) || !aligned_ptr(z, 16) || !aligned_ptr(weight, 16) || !aligned_ptr(y, 16) ||
        !aligned_ptr(scales, 4))
        return KKT_ERR_ALIGN;
    if (rows == 0) return KKT_OK;
    NormParams p;
    p.x = x; p.r = nullptr; p.z = z; p.w = weight; p.y = y; p.r_out = nullptr; p.scales = scales;
    p.rows = rows; p.dim = dim; p.group = 0; p.eps = eps;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return io_dtype == KKT_IO_BF16 ? launch_gated<__nv_bfloat16>(p, out_dtype, st)
                                   : launch_gated<float>(p, out_dtype, st);
}
