// gdn_recurrent.cu -- the gated delta rule token by token over a pool of states: gdn_recurrent_fwd
// (include/gdn_layer.h), the decode form of the chunk recurrence in gdn_chunk.cu.
//
// Per sequence and value head, with S (dk x dv) in fp32 registers for the whole call:
//     z = S^T k,  y = S^T q                                (one pass over S)
//     d = beta (v - a z),   S <- a S + k d^T,   o = scale (a y + (k . q) d)
// which is the rule with o = scale S_new^T q expanded, so that a token needs one reduction over the
// rows of S instead of two.
//
// The columns of S are independent.  A warp owns 16 of them: lane = 4 r + c holds columns 4c .. 4c+3
// of the rows DK/8 r .. DK/8 (r + 1) - 1, so a row's 16 columns are one 64-byte segment, and the
// reductions over the rows are in-register sums and three shuffles.  A block is one (sequence, head),
// its warps the column slabs; no shared memory and no barrier.
#include "gdn_layer.cuh"

namespace kkt {
namespace {

using namespace ptx;

struct RecParams {
    const void *q, *k, *v;
    const float *beta, *g;
    const int32_t *cu, *slots, *slots_out;
    void *state, *o;
    int N, T, Hk, Hv, num_slots;
    int64_t ntok;
    float scale;
    int *status;
};

// R consecutive values as fp32 (R a multiple of 8).
template <int R, typename T>
__device__ __forceinline__ void load_rows(const T *p, float (&v)[R]) {
#pragma unroll
    for (int i = 0; i < R; i += 8) {
        float w[8];
        widen8(raw8(p + i), w);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i + e] = w[e];
    }
}

template <typename IO, typename ST, int DK, int DV>
__global__ void __launch_bounds__(2 * DV) gdn_recurrent_kernel(const RecParams p) {
    constexpr int R = DK / 8;
    griddep_launch_dependents();
    griddep_wait();
    const int n = blockIdx.x / p.Hv, h = blockIdx.x % p.Hv;
    const int lane = threadIdx.x & 31;
    const int row0 = (lane >> 2) * R;
    const int col = (threadIdx.x >> 5) * 16 + (lane & 3) * 4;
    Span s = seq_span(p.cu, n, p.N, p.T, p.ntok, p.status);
    const int in = slot_of(p.slots, n, p.num_slots, p.status, s.ok);
    const int out = p.slots_out ? slot_of(p.slots_out, n, p.num_slots, p.status, s.ok) : in;
    if (!s.ok) return;
    const int64_t off = ((int64_t)h * DK + row0) * DV + col;
    const int64_t slot_size = (int64_t)p.Hv * DK * DV;

    float S[R][4];
    const ST *src = static_cast<const ST *>(p.state) + in * slot_size + off;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const float4 x = in >= 0 ? load4(src + i * DV) : make_float4(0.f, 0.f, 0.f, 0.f);
        S[i][0] = x.x; S[i][1] = x.y; S[i][2] = x.z; S[i][3] = x.w;
    }
    const int hk = h / (p.Hv / p.Hk);
    const IO *q = static_cast<const IO *>(p.q) + hk * DK + row0;
    const IO *k = static_cast<const IO *>(p.k) + hk * DK + row0;
    for (int64_t t = s.a; t < s.b; ++t) {
        float kv[R], qv[R];
        load_rows(k + t * p.Hk * DK, kv);
        load_rows(q + t * p.Hk * DK, qv);
        const int64_t tv = t * p.Hv + h;
        const float4 v = load4(static_cast<const IO *>(p.v) + tv * DV + col);
        const float beta = __ldg(p.beta + tv);
        const float a = p.g ? expf(__ldg(p.g + tv)) : 1.f;
        float z[4] = {0.f, 0.f, 0.f, 0.f}, y[4] = {0.f, 0.f, 0.f, 0.f}, kq = 0.f;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            kq = fmaf(kv[i], qv[i], kq);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                z[c] = fmaf(S[i][c], kv[i], z[c]);
                y[c] = fmaf(S[i][c], qv[i], y[c]);
            }
        }
#pragma unroll
        for (int m = 4; m < 32; m <<= 1) {
            kq += __shfl_xor_sync(0xffffffffu, kq, m);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                z[c] += __shfl_xor_sync(0xffffffffu, z[c], m);
                y[c] += __shfl_xor_sync(0xffffffffu, y[c], m);
            }
        }
        const float vv[4] = {v.x, v.y, v.z, v.w};
        float d[4], ov[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            d[c] = beta * (vv[c] - a * z[c]);
            ov[c] = p.scale * fmaf(kq, d[c], a * y[c]);
        }
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) S[i][c] = fmaf(kv[i], d[c], a * S[i][c]);
        if (lane < 4) store4(static_cast<IO *>(p.o) + tv * DV + col, make_float4(ov[0], ov[1], ov[2], ov[3]));
    }
    if (out >= 0 && (out != in || s.b > s.a)) {
        ST *dst = static_cast<ST *>(p.state) + out * slot_size + off;
#pragma unroll
        for (int i = 0; i < R; ++i) store4(dst + i * DV, make_float4(S[i][0], S[i][1], S[i][2], S[i][3]));
    }
}

template <typename IO, typename ST>
int launch(const RecParams &p, int dk, int dv, cudaStream_t st) {
    const dim3 grid((unsigned)(p.N * p.Hv));
    if (dk == 128)
        return dv == 128 ? launch_serialised(gdn_recurrent_kernel<IO, ST, 128, 128>, grid, 256, 0, st, p)
                         : launch_serialised(gdn_recurrent_kernel<IO, ST, 128, 64>, grid, 128, 0, st, p);
    return dv == 128 ? launch_serialised(gdn_recurrent_kernel<IO, ST, 64, 128>, grid, 256, 0, st, p)
                     : launch_serialised(gdn_recurrent_kernel<IO, ST, 64, 64>, grid, 128, 0, st, p);
}

}  // namespace
}  // namespace kkt

extern "C" int gdn_recurrent_fwd(const void *q, const void *k, const void *v, const float *beta, const float *g,
                                 const int32_t *cu_seqlens, int N, int T, int Hk, int Hv, int dk, int dv, float scale,
                                 int io_dtype, void *state, int state_dtype, int num_slots, const int32_t *slots,
                                 const int32_t *slots_out, void *o, struct CUstream_st *stream) {
    using namespace kkt;
    if (N < 1 || T < 0 || Hk < 1 || Hv < 1 || Hv > 65535 || Hv % Hk != 0 || num_slots < 0) return KKT_ERR_ARG;
    if ((io_dtype != KKT_IO_BF16 && io_dtype != KKT_IO_F32) || (state_dtype != KKT_IO_BF16 && state_dtype != KKT_IO_F32))
        return KKT_ERR_ARG;
    if ((dk != 64 && dk != 128) || (dv != 64 && dv != 128)) return KKT_ERR_UNSUPPORTED;
    const int64_t ntok = cu_seqlens ? (int64_t)T : (int64_t)N * T;
    if (ntok > 0x7fffffffLL || (int64_t)N * Hv > 0x7fffffffLL) return KKT_ERR_ARG;
    if (ntok > 0 && (!q || !k || !v || !beta || !o)) return KKT_ERR_ARG;
    if (num_slots > 0 && !state) return KKT_ERR_ARG;
    if (!slots && N > num_slots) return KKT_ERR_ARG;
    if (!aligned_ptr(q, 16) || !aligned_ptr(k, 16) || !aligned_ptr(v, 16) || !aligned_ptr(o, 16) ||
        !aligned_ptr(state, 16) || !aligned_ptr(beta, 4) || !aligned_ptr(g, 4) || !aligned_ptr(cu_seqlens, 4) ||
        !aligned_ptr(slots, 4) || !aligned_ptr(slots_out, 4))
        return KKT_ERR_ALIGN;
    if (ntok == 0 && !slots_out && !cu_seqlens) return KKT_OK;  // every state stays where it is
    RecParams p;
    p.q = q; p.k = k; p.v = v; p.beta = beta; p.g = g;
    p.cu = cu_seqlens; p.slots = slots; p.slots_out = slots_out;
    p.state = state; p.o = o;
    p.N = N; p.T = T; p.Hk = Hk; p.Hv = Hv; p.num_slots = num_slots;
    p.ntok = ntok; p.scale = scale;
    const int rc = status_ptr(&p.status);
    if (rc != KKT_OK) return rc;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (io_dtype == KKT_IO_BF16)
        return state_dtype == KKT_IO_BF16 ? launch<__nv_bfloat16, __nv_bfloat16>(p, dk, dv, st)
                                          : launch<__nv_bfloat16, float>(p, dk, dv, st);
    return state_dtype == KKT_IO_BF16 ? launch<float, __nv_bfloat16>(p, dk, dv, st)
                                      : launch<float, float>(p, dk, dv, st);
}
