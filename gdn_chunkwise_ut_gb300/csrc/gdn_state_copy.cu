// gdn_state_copy.cu -- copies and clears pool slots of many tensors in one launch: gdn_state_copy
// (include/gdn_layer.h).
//
// A block moves one piece of 16 KB of one slot of one tensor; the pieces of all tensors are one axis of
// the grid, so that small tensors beside large ones leave no block empty (with an axis for the tensors,
// 201 us in the case below).  Bound by HBM: 61 moves and 19 clears in the pools of four layers, 1.21 GB,
// take 172.5 us, 105% of the copy rate; four copies of one slot in two layers 3.9 us, launch and latency.
#include "gdn_layer.cuh"

namespace kkt {
namespace {

using namespace ptx;

constexpr int kCopyThreads = 256;
constexpr int kCopyLoads = 4;  // 16-byte vectors of a thread, all loaded before the first is stored
constexpr size_t kCopyPiece = (size_t)kCopyThreads * kCopyLoads * 16;

struct CopyTensor {
    uint8_t *dst;
    const uint8_t *src;
    size_t bytes, dst_stride, src_stride;
};
struct CopyParams {
    CopyTensor t[GDN_COPY_MAX_TENSORS];
    unsigned end[GDN_COPY_MAX_TENSORS];  // pieces of a move up to and with tensor i
    const int32_t *dst_slots, *src_slots;
    int dst_num, src_num;
    int *status;
};

__global__ void __launch_bounds__(kCopyThreads) state_copy_kernel(const __grid_constant__ CopyParams p) {
    griddep_launch_dependents();
    griddep_wait();
    int i = 0;
    while (blockIdx.x >= p.end[i]) ++i;  // blockIdx.x is below the last tensor's end
    const CopyTensor &t = p.t[i];
    const size_t first = (size_t)(blockIdx.x - (i ? p.end[i - 1] : 0u)) * kCopyPiece;
    const int m = blockIdx.y;
    const int d = p.dst_slots[m];
    const int s = p.src_slots ? p.src_slots[m] : -1;
    if (d >= p.dst_num || s >= p.src_num) {
        record_error(p.status, KKT_ERR_INDEX);
        return;
    }
    if (d < 0) return;
    uint8_t *dst = t.dst + (size_t)d * t.dst_stride;
    const uint8_t *src = s >= 0 ? t.src + (size_t)s * t.src_stride : nullptr;
    const size_t last = first + kCopyPiece < t.bytes ? first + kCopyPiece : t.bytes;
    const bool wide = ((reinterpret_cast<uintptr_t>(dst) | reinterpret_cast<uintptr_t>(src) | t.bytes) & 15) == 0;
    if (wide) {
        uint4 v[kCopyLoads];
#pragma unroll
        for (int i = 0; i < kCopyLoads; ++i) {
            const size_t at = first + (threadIdx.x + (size_t)i * kCopyThreads) * 16;
            v[i] = src && at < last ? *reinterpret_cast<const uint4 *>(src + at) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < kCopyLoads; ++i) {
            const size_t at = first + (threadIdx.x + (size_t)i * kCopyThreads) * 16;
            if (at < last) *reinterpret_cast<uint4 *>(dst + at) = v[i];
        }
    } else {
        for (size_t at = first + threadIdx.x; at < last; at += kCopyThreads) dst[at] = src ? src[at] : 0;
    }
}

}  // namespace
}  // namespace kkt

extern "C" int gdn_state_copy(void *const *dst, const void *const *src, const size_t *slot_bytes,
                              const size_t *dst_stride, const size_t *src_stride, int ntensors,
                              const int32_t *dst_slots, const int32_t *src_slots, int nmoves, int dst_num_slots,
                              int src_num_slots, struct CUstream_st *stream) {
    using namespace kkt;
    if (ntensors < 1 || ntensors > GDN_COPY_MAX_TENSORS || nmoves < 0 || dst_num_slots < 0 || src_num_slots < 0)
        return KKT_ERR_ARG;
    if (!dst || !slot_bytes || !dst_stride || (src && (!src_stride || (nmoves > 0 && !src_slots))))
        return KKT_ERR_ARG;
    if (nmoves > 0 && !dst_slots) return KKT_ERR_ARG;
    if (!aligned_ptr(dst_slots, 4) || !aligned_ptr(src_slots, 4)) return KKT_ERR_ALIGN;
    CopyParams p = {};
    size_t pieces = 0;  // of a move
    for (int i = 0; i < ntensors; ++i) {
        if ((dst_num_slots > 0 && !dst[i]) || (src && src_num_slots > 0 && !src[i])) return KKT_ERR_ARG;
        // slots of a tensor do not overlap
        if (slot_bytes[i] < 1 || dst_stride[i] < slot_bytes[i] || (src && src_stride[i] < slot_bytes[i]))
            return KKT_ERR_ARG;
        p.t[i].dst = static_cast<uint8_t *>(dst[i]);
        p.t[i].src = src ? static_cast<const uint8_t *>(src[i]) : nullptr;
        p.t[i].bytes = slot_bytes[i];
        p.t[i].dst_stride = dst_stride[i];
        p.t[i].src_stride = src ? src_stride[i] : 0;
        pieces += (slot_bytes[i] + kCopyPiece - 1) / kCopyPiece;
        if (slot_bytes[i] > SIZE_MAX / 2 || pieces > 0x7fffffffu) return KKT_ERR_ARG;
        p.end[i] = (unsigned)pieces;
    }
    p.dst_num = dst_num_slots;
    p.src_num = src_num_slots;
    const int rc = nmoves > 0 ? status_ptr(&p.status) : KKT_OK;
    if (rc != KKT_OK) return rc;
    constexpr int kMostMoves = 65535;  // of one launch: the grid's second dimension
    for (int m = 0; m < nmoves; m += kMostMoves) {
        p.dst_slots = dst_slots + m;
        p.src_slots = src ? src_slots + m : nullptr;  // without sources every slot is cleared
        const dim3 grid((unsigned)pieces, (unsigned)(nmoves - m < kMostMoves ? nmoves - m : kMostMoves));
        const int e = launch_serialised(state_copy_kernel, grid, kCopyThreads, 0,
                                        reinterpret_cast<cudaStream_t>(stream), p);
        if (e != KKT_OK) return e;
    }
    return KKT_OK;
}
