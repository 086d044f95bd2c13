// gdn_prep.cu -- from a layer's projections to the delta rule's q, k, v, g and beta: gdn_prep_fwd
// (include/gdn_layer.h).  One pass over the packed channels: the short causal convolution along the
// tokens, SiLU, and for q and k the L2 norm of each head.
//
// A warp owns a slab of 256 consecutive channels (8 to a lane, 16 bytes of bf16: whole heads, since a
// head is 64 or 128 channels) of a run of consecutive tokens, and keeps the last three inputs of its
// channels in registers, so a run reads every input once (plus three before its first token).  A
// head's sum of squares is a shuffle over its 8 or 16 lanes.  The two gates are one more slab.
//
// The convolution's state is read, and its successor written, by the warp that has the sequence's
// first token, whichever run holds the last one: the same thread reads and writes each element, so
// updating the pool in place needs no order between warps.  For that, the tokens whose window reaches
// into the state belong to that warp too: a run goes on over them past its end, and the next one
// leaves them out.
#include "gdn_layer.cuh"

namespace kkt {
namespace {

using namespace ptx;

constexpr int kPrepWarps = 8;
constexpr int kPrepBatch = 4;  // tokens whose inputs are loaded together
constexpr int kSlab = 256;     // channels of a warp

struct PrepParams {
    const void *x, *weight, *bias, *a, *b;
    const float *A_log, *dt_bias;
    const int32_t *cu, *slots;
    void *conv_state, *q, *k, *v;
    float *g, *beta;
    int N, T, Hk, Hv, D, taps, expand, run, num_slots, slabs;
    int64_t ntok;
    float eps;
    int *status;
};

// The sequence of token t: the last one that starts at or before it (empty ones before it are passed
// over).  False, with the error recorded, where cu_seqlens is malformed there.
__device__ __forceinline__ bool seq_of_token(const PrepParams &p, int64_t t, int &n, int64_t &a, int64_t &b) {
    if (!p.cu) {
        n = (int)(t / p.T);
        a = (int64_t)n * p.T;
        b = a + p.T;
        return true;
    }
    int lo = 0, hi = p.N - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (__ldg(p.cu + mid) <= t) lo = mid; else hi = mid - 1;
    }
    n = lo;
    const Span s = seq_span(p.cu, n, p.N, p.T, p.ntok, p.status);
    a = s.a;
    b = s.b;
    if (s.ok && (t < a || t >= b)) {
        record_error(p.status, KKT_ERR_SEQLENS);
        return false;
    }
    return s.ok;
}

// beta = sigmoid(b) and g = -e^{A_log} softplus(a + dt_bias) of `count` consecutive (token, head) pairs.
template <typename IO>
__device__ __forceinline__ void gates(const PrepParams &p, int64_t first, int64_t count, int lane) {
    for (int64_t i = first + lane; i < first + count; i += 32) {
        const int h = (int)(i % p.Hv);
        const float bb = to_f32(static_cast<const IO *>(p.b)[i]);
        const float u = to_f32(static_cast<const IO *>(p.a)[i]) + __ldg(p.dt_bias + h);
        p.beta[i] = 1.f / (1.f + expf(-bb));
        // softplus(u) = max(u, 0) + log(1 + e^-|u|); a NaN stays one
        p.g[i] = -expf(__ldg(p.A_log + h)) * ((u > 0.f ? u : u < 0.f ? 0.f : u) + log1pf(expf(-fabsf(u))));
    }
}

template <typename IO, int DH>
__global__ void __launch_bounds__(kPrepWarps * 32) gdn_prep_kernel(const PrepParams p) {
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const int slab = blockIdx.y * kPrepWarps + (threadIdx.x >> 5);
    const int64_t t0 = (int64_t)blockIdx.x * p.run;
    const int64_t t1 = t0 + p.run < p.ntok ? t0 + p.run : p.ntok;
    if (slab > p.slabs) return;
    if (slab == p.slabs) {
        gates<IO>(p, t0 * p.Hv, (t1 - t0) * p.Hv, lane);
        if (blockIdx.x == 0 && p.cu)
            for (int n = lane; n < p.N; n += 32) check_sequence(p.cu, n, p.N, p.ntok, p.status);
        return;
    }
    const int ch = slab * kSlab + lane * 8;
    const bool live = ch < p.D;  // the last slab may be short
    const int chc = live ? ch : 0;
    const int keep = p.taps - 1;

    // weights, in front of them zeros where there are fewer than four taps
    float w[4][8], bias[8];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int tap = j - (4 - p.taps);
            w[j][e] = tap >= 0 ? to_f32(static_cast<const IO *>(p.weight)[(int64_t)(chc + e) * p.taps + tap]) : 0.f;
        }
#pragma unroll
    for (int e = 0; e < 8; ++e) bias[e] = p.bias ? to_f32(static_cast<const IO *>(p.bias)[chc + e]) : 0.f;

    // where this lane's head goes
    const int head = chc / DH;
    const bool norm = head < 2 * p.Hk;
    const int rep = p.Hv / p.Hk;
    IO *dst;
    int64_t dst_stride;
    int copies = 1;
    if (norm) {
        const int j = head < p.Hk ? head : head - p.Hk;
        dst = static_cast<IO *>(head < p.Hk ? p.q : p.k);
        const int ho = p.expand ? j * rep : j;
        dst_stride = (int64_t)(p.expand ? p.Hv : p.Hk) * DH;
        dst += (int64_t)ho * DH + chc % DH;
        if (p.expand) copies = rep;
    } else {
        dst = static_cast<IO *>(p.v) + (int64_t)(head - 2 * p.Hk) * DH + chc % DH;
        dst_stride = (int64_t)p.Hv * DH;
    }

    const IO *x = static_cast<const IO *>(p.x) + chc;
    float win[3][8];  // the three inputs before the current token, oldest first
#pragma unroll
    for (int j = 0; j < 3; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) win[j][e] = 0.f;

    int n = 0;
    int64_t a = 0, b = -1;
    int slot = -1;
    bool ok = false;
    int64_t t = t0, end = t1;
    if (keep > 1 && seq_of_token(p, t0, n, a, b) && t0 > a && t0 < a + keep) t = a + keep < b ? a + keep : b;
    b = -1;  // the loop looks its first token up itself
    while (t < end) {
        const int count = end - t < kPrepBatch ? (int)(end - t) : kPrepBatch;
        Raw8<IO> in[kPrepBatch];
#pragma unroll
        for (int i = 0; i < kPrepBatch; ++i)
            if (i < count) in[i] = raw8(x + (t + i) * p.D);
#pragma unroll
        for (int i = 0; i < kPrepBatch; ++i) {
            if (i >= count) break;
            const int64_t tt = t + i;
            if (tt >= b) {
                // a new sequence (or the run's first token): the inputs before it
                ok = seq_of_token(p, tt, n, a, b);
                if (!ok) b = tt + 1;  // this token alone is passed over
                slot = -1;
                if (ok) slot = slot_of(p.slots, n, p.num_slots, p.status, ok);
                if (ok) {
                    const int64_t pos = tt - a;
                    IO *state = static_cast<IO *>(p.conv_state) + (int64_t)slot * keep * p.D + chc;
#pragma unroll
                    for (int j = 0; j < 3; ++j) {
                        const int back = 3 - j;  // the input `back` tokens before this one
#pragma unroll
                        for (int e = 0; e < 8; ++e) win[j][e] = 0.f;
                        if (back <= keep) {
                            if (pos >= back) widen8(raw8(x + (tt - back) * p.D), win[j]);
                            else if (slot >= 0) widen8(raw8(state + (keep + pos - back) * p.D), win[j]);
                        }
                    }
                    if (pos == 0 && a + keep > t1 && b > t1) end = a + keep < b ? a + keep : b;
                    if (pos == 0 && slot >= 0 && live) {
                        // the state the sequence leaves: the last `keep` of the old state and its inputs,
                        // oldest first, so that an old row is read before it is overwritten
                        const int64_t len = b - a;
                        for (int r = 0; r < keep; ++r) {
                            const int64_t from = len + r;
                            const Raw8<IO> row = from < keep ? raw8(state + from * p.D) : raw8(x + (a + from - keep) * p.D);
                            float f[8];
                            widen8(row, f);
                            store8(state + (int64_t)r * p.D, f);
                        }
                    }
                }
            }
            float cur[8], y[8];
            widen8(in[i], cur);
            float ss = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float acc = fmaf(win[0][e], w[0][e], bias[e]);
                acc = fmaf(win[1][e], w[1][e], acc);
                acc = fmaf(win[2][e], w[2][e], acc);
                acc = fmaf(cur[e], w[3][e], acc);
                y[e] = silu(acc);
                ss = fmaf(y[e], y[e], ss);
                win[0][e] = win[1][e];
                win[1][e] = win[2][e];
                win[2][e] = cur[e];
            }
            ss = lanes_sum<DH / 8>(ss);
            if (norm) {
                const float r = rsqrtf(ss + p.eps);
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] *= r;
            }
            if (live && ok) {
                IO *o = dst + tt * dst_stride;
                for (int c = 0; c < copies; ++c) store8(o + c * DH, y);
            }
        }
        t += count;
    }
}

template <typename IO>
int launch(PrepParams &p, int dh, cudaStream_t st) {
    p.slabs = (p.D + kSlab - 1) / kSlab;
    // Tokens of a run: a longer run re-reads fewer of the three inputs before it, a shorter one gives
    // more warps.  16 (19% re-reads, from the caches) once that leaves 8 warps for every SM.
    const int64_t want = (int64_t)sm_count_cached() * 8;
    p.run = 16;
    while (p.run > 1 && (p.ntok + p.run - 1) / p.run * (p.slabs + 1) < want) p.run /= 4;
    const dim3 grid((unsigned)((p.ntok + p.run - 1) / p.run), (unsigned)((p.slabs + 1 + kPrepWarps - 1) / kPrepWarps));
    return dh == 128 ? launch_serialised(gdn_prep_kernel<IO, 128>, grid, kPrepWarps * 32, 0, st, p)
                     : launch_serialised(gdn_prep_kernel<IO, 64>, grid, kPrepWarps * 32, 0, st, p);
}

}  // namespace
}  // namespace kkt

extern "C" int gdn_prep_fwd(const void *x, const void *weight, const void *bias, const void *a, const void *b,
                            const float *A_log, const float *dt_bias, const int32_t *cu_seqlens, int N, int T, int Hk,
                            int Hv, int dk, int dv, int taps, float eps, int expand, int io_dtype, void *conv_state,
                            int num_slots, const int32_t *slots, void *q, void *k, void *v, float *g, float *beta,
                            struct CUstream_st *stream) {
    using namespace kkt;
    if (N < 1 || T < 0 || Hk < 1 || Hv < 1 || Hv > 65535 || Hv % Hk != 0 || num_slots < 0) return KKT_ERR_ARG;
    if (io_dtype != KKT_IO_BF16 && io_dtype != KKT_IO_F32) return KKT_ERR_ARG;
    if (dk != dv || (dk != 64 && dk != 128) || taps < 2 || taps > 4) return KKT_ERR_UNSUPPORTED;
    const int64_t ntok = cu_seqlens ? (int64_t)T : (int64_t)N * T;
    const int64_t D = ((int64_t)2 * Hk + Hv) * dk;
    if (ntok > 0x7fffffffLL || D > (int64_t)kSlab * 65535) return KKT_ERR_ARG;
    if (!weight || !A_log || !dt_bias) return KKT_ERR_ARG;
    if (ntok > 0 && (!x || !a || !b || !q || !k || !v || !g || !beta)) return KKT_ERR_ARG;
    if (num_slots > 0 && !conv_state) return KKT_ERR_ARG;
    if (!slots && N > num_slots) return KKT_ERR_ARG;
    const int es = io_dtype == KKT_IO_BF16 ? 2 : 4;
    if (!aligned_ptr(x, 16) || !aligned_ptr(weight, es) || !aligned_ptr(bias, es) || !aligned_ptr(a, es) ||
        !aligned_ptr(b, es) || !aligned_ptr(A_log, 4) || !aligned_ptr(dt_bias, 4) || !aligned_ptr(cu_seqlens, 4) ||
        !aligned_ptr(slots, 4) || !aligned_ptr(conv_state, 16) || !aligned_ptr(q, 16) || !aligned_ptr(k, 16) ||
        !aligned_ptr(v, 16) || !aligned_ptr(g, 4) || !aligned_ptr(beta, 4))
        return KKT_ERR_ALIGN;
    if (ntok == 0) return KKT_OK;
    PrepParams p;
    p.x = x; p.weight = weight; p.bias = bias; p.a = a; p.b = b;
    p.A_log = A_log; p.dt_bias = dt_bias; p.cu = cu_seqlens; p.slots = slots;
    p.conv_state = conv_state; p.q = q; p.k = k; p.v = v; p.g = g; p.beta = beta;
    p.N = N; p.T = T; p.Hk = Hk; p.Hv = Hv; p.D = (int)D; p.taps = taps; p.expand = expand != 0;
    p.num_slots = num_slots; p.ntok = ntok; p.eps = eps;
    const int rc = status_ptr(&p.status);
    if (rc != KKT_OK) return rc;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return io_dtype == KKT_IO_BF16 ? launch<__nv_bfloat16>(p, dk, st) : launch<float>(p, dk, st);
}
