// gfx950 kernels of the low-precision weight codecs and the C ABI that
// launches them (declared in include/lpq.h).
//
// Formats ("Low Precision RL", "Choose a precision"; "verl NVFP4 QAT",
// sections 2.3-2.5 and 3.3): block-wise FP8 (E4M3, FP32 scale per 128x128
// tile), MXFP8 (E4M3, UE8M0 byte per 1x32 block) and NVFP4 (E2M1, E4M3 scale
// per 1x16 block, FP32 global scale amax / 2688 shared by a sibling group),
// plus the NVFP4 fake-quant; MXFP4 (E2M1, UE8M0 byte per 1x32 block).  The
// codecs are streaming work bound by HBM bandwidth, and so are the two-way
// quantizer and the root-mean-square norm of the quantized layer; its products
// run on the matrix cores (lpq_mx_matmul.hpp).
//
// Launch shape.  A grouped call covers many tensors in one launch.  The grid
// is one-dimensional and dense: the host lays the tensors' work units
// (chunks, or 128x128 tiles) end to end and passes a short table of
// equal-size runs in the kernel arguments; each workgroup finds its tensor
// from that table with scalar compares and one division, then reads the
// descriptor into scalar registers.
// No workgroup is launched without work.
//  * MXFP8 / MXFP4 / NVFP4 / INT4 are flat in memory (N is a multiple of the block),
//    so a workgroup (128, 256 or 512 threads, chosen per kernel) streams
//    16-byte BF16 vectors, 8 elements per lane, U vectors per lane; a 1x32 block is a quad of lanes and a 1x16 block a pair,
//    reduced with DPP lane permutations.  U is 2 to 4 (16 for the read-only
//    amax pass): enough bytes in flight per CU, short-lived workgroups.  A
//    lane's U loads go out either all at once or one vector ahead of the
//    work, chosen per kernel by measurement: the encoders and the MXFP8
//    decoder run faster with fewer reads in flight per wave.  Full chunks
//    (all but a tensor's last) take a body compiled without bounds checks.
//  * Block-wise FP8 quantization gives one workgroup a strip of 2 or 4
//    adjacent 128x128 tiles (one per 256 threads): 16 lanes per 256-byte row
//    segment of a tile, 8 row passes, all values kept in registers between the
//    per-tile amax reduction (DPP + LDS across the waves) and the encode, so
//    HBM is read once.  Dequantization streams flat when the layout allows,
//    else one tile per workgroup.
#include <hip/hip_runtime.h>
#include <hip/hip_bf16.h>
#include <stdint.h>

#include <atomic>
#include <type_traits>

#include "lpq.h"
#include "lpq_device.hpp"

// Launch parameters, then the kernels, format by format.
#include "lpq_tuning.hpp"

using namespace lpq;

#include "lpq_flat.hpp"
#include "lpq_mxfp8.hpp"
#include "lpq_mxfp4.hpp"
#include "lpq_nvfp4.hpp"
#include "lpq_int4.hpp"
#include "lpq_fp8blk.hpp"
#include "lpq_requant.hpp"
#include "lpq_mx_transpose.hpp"
#include "lpq_rmsnorm.hpp"
#include "lpq_mx_matmul.hpp"


// ===========================================================================
// Host side: argument checks and launches
// ===========================================================================

namespace {

thread_local int g_last_hip_error = 0;

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline lpq_status launched() {
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) {
        g_last_hip_error = (int)e;
        return LPQ_ERR_HIP;
    }
    return LPQ_OK;
}

enum Kind {
    FP8BLK_Q, FP8BLK_QW, FP8BLK_DQ, FP8BLK_DQF, MXFP8_Q, MXFP8_QF, MXFP8_DQ,
    MXFP4_Q, MXFP4_QF, MXFP4_DQ, MXFP4_QDQ, MXFP4_QDQF, NV_AMAX, NV_Q, NV_DQ, NV_QDQ, NV_QDQ_W,
    I4_Q32, I4_Q128, I4_DQ32, I4_DQ128, I4_QDQ32, I4_QDQ128,
    RQ_FP8, RQ_MX, RQ_AMAX, RQ_NV
};

// The INT4 group size of an INT4 kind (0 for other kinds).
constexpr int int4_group(Kind k) {
    return (k == I4_Q32 || k == I4_DQ32 || k == I4_QDQ32) ? 32 : (k == I4_Q128 || k == I4_DQ128 || k == I4_QDQ128) ? 128 : 0;
}

// Shape and pointer checks of one tensor for one kind of call.
int64_t units(Kind k, const lpq_tensor& t);
int64_t units(Kind k, const lpq_requant_tensor& t);
bool one_launch_holds(Kind k, int64_t units);

lpq_status check_tensor(Kind k, const lpq_tensor& t, int32_t n_groups) {
    if (t.rows <= 0 || t.cols <= 0) return LPQ_ERR_SHAPE;
    if (t.rows > (int64_t(1) << 40) / t.cols) return LPQ_ERR_SHAPE;   // element count overflow guard
    if (!t.src) return LPQ_ERR_NULL;
    if (k != NV_AMAX && !t.dst) return LPQ_ERR_NULL;
    if (k != NV_AMAX && k != NV_QDQ && k != I4_QDQ32 && k != I4_QDQ128 && k != MXFP4_QDQ && k != MXFP4_QDQF && !t.scale)
        return LPQ_ERR_NULL;
    if (t.reserved != 0) return LPQ_ERR_ARG;
    switch (k) {
    case FP8BLK_Q:
    case FP8BLK_QW:   // not a caller-visible kind: the wide-strip quantizer
    case FP8BLK_DQ:
        if (!aligned(k == FP8BLK_DQ ? t.dst : t.src, 2) || !aligned(t.scale, 4)) return LPQ_ERR_ALIGN;
        break;
    case FP8BLK_DQF:   // not a caller-visible kind: the flat layout's extra conditions
        if (t.cols % 8 || t.rows >= (int64_t(1) << 31) || t.cols >= (int64_t(1) << 31) - kRqStepMax) return LPQ_ERR_SHAPE;
        if (!aligned(t.src, 8) || !aligned(t.dst, 16) || !aligned(t.scale, 4)) return LPQ_ERR_ALIGN;
        break;
    case MXFP8_Q:
    case MXFP8_QF:
        if (t.cols % 32) return LPQ_ERR_SHAPE;
        if (!aligned(t.src, 16) || !aligned(t.dst, 8)) return LPQ_ERR_ALIGN;
        break;
    case MXFP8_DQ:
        if (t.cols % 32) return LPQ_ERR_SHAPE;
        if (!aligned(t.src, 8) || !aligned(t.dst, 16)) return LPQ_ERR_ALIGN;
        break;
    case MXFP4_Q:
    case MXFP4_QF:
        if (t.cols % 32) return LPQ_ERR_SHAPE;
        if (!aligned(t.src, 16) || !aligned(t.dst, 4)) return LPQ_ERR_ALIGN;
        break;
    case MXFP4_DQ:
        if (t.cols % 32) return LPQ_ERR_SHAPE;
        if (!aligned(t.src, 4) || !aligned(t.dst, 16)) return LPQ_ERR_ALIGN;
        break;
    case MXFP4_QDQ:
    case MXFP4_QDQF:
        if (t.cols % 32) return LPQ_ERR_SHAPE;
        if (!aligned(t.src, 16) || !aligned(t.dst, 16)) return LPQ_ERR_ALIGN;
        break;
    case NV_AMAX:
    case NV_Q:
    case NV_DQ:
    case NV_QDQ:
        if (t.cols % 16) return LPQ_ERR_SHAPE;
        if (k == NV_DQ ? !aligned(t.src, 4) : !aligned(t.src, 16)) return LPQ_ERR_ALIGN;
        if (k == NV_Q && !aligned(t.dst, 4)) return LPQ_ERR_ALIGN;
        if ((k == NV_DQ || k == NV_QDQ) && !aligned(t.dst, 16)) return LPQ_ERR_ALIGN;
        if (n_groups > 0 && (t.group < 0 || t.group >= n_groups)) return LPQ_ERR_GROUP;
        break;
    case I4_Q32:
    case I4_Q128:
        if (t.cols % int4_group(k)) return LPQ_ERR_SHAPE;
        if (!aligned(t.src, 16) || !aligned(t.dst, 4) || !aligned(t.scale, 4)) return LPQ_ERR_ALIGN;
        break;
    case I4_DQ32:
    case I4_DQ128:
        if (t.cols % int4_group(k)) return LPQ_ERR_SHAPE;
        if (!aligned(t.src, 4) || !aligned(t.dst, 16) || !aligned(t.scale, 4)) return LPQ_ERR_ALIGN;
        break;
    case I4_QDQ32:
    case I4_QDQ128:
        if (t.cols % int4_group(k)) return LPQ_ERR_SHAPE;
        if (!aligned(t.src, 16) || !aligned(t.dst, 16)) return LPQ_ERR_ALIGN;
        break;
    default: return LPQ_ERR_ARG;
    }
    return one_launch_holds(k, units(k, t)) ? LPQ_OK : LPQ_ERR_SHAPE;
}

lpq_status check_tensor(Kind k, const lpq_requant_tensor& t, int32_t n_groups) {
    if (t.rows <= 0 || t.cols <= 0) return LPQ_ERR_SHAPE;
    if (t.rows > (int64_t(1) << 40) / t.cols) return LPQ_ERR_SHAPE;
    if (!t.src || !t.src_scale) return LPQ_ERR_NULL;
    if (k != RQ_AMAX && (!t.dst || !t.dst_scale)) return LPQ_ERR_NULL;
    if (t.reserved != 0) return LPQ_ERR_ARG;
    if (!one_launch_holds(k, units(k, t))) return LPQ_ERR_SHAPE;
    if (k == RQ_FP8) return aligned(t.src_scale, 4) && aligned(t.dst_scale, 4) ? LPQ_OK : LPQ_ERR_ALIGN;
    if (t.cols % (k == RQ_MX ? 32 : 16)) return LPQ_ERR_SHAPE;
    if (t.rows >= (int64_t(1) << 31) || t.cols >= (int64_t(1) << 31) - kRqStepMax) return LPQ_ERR_SHAPE;
    if (!aligned(t.src, 16) || !aligned(t.src_scale, 4)) return LPQ_ERR_ALIGN;
    if (k == RQ_MX && !aligned(t.dst, 16)) return LPQ_ERR_ALIGN;
    if (k == RQ_NV && !aligned(t.dst, 8)) return LPQ_ERR_ALIGN;
    if (k != RQ_MX && n_groups > 0 && (t.group < 0 || t.group >= n_groups)) return LPQ_ERR_GROUP;
    return LPQ_OK;
}

// Work units (workgroups) of one tensor.
int64_t units(Kind k, const lpq_tensor& t) {
    const int64_t n = t.rows * t.cols;
    switch (k) {
    case FP8BLK_Q: return ((t.rows + kTile - 1) / kTile) * ((t.cols + kTile * LPQ_TILEQ_TW - 1) / (kTile * LPQ_TILEQ_TW));
    case FP8BLK_QW:
        return ((t.rows + kTile - 1) / kTile) * ((t.cols + kTile * LPQ_TILEQ_WIDE_TW - 1) / (kTile * LPQ_TILEQ_WIDE_TW));
    case FP8BLK_DQ: return ((t.rows + kTile - 1) / kTile) * ((t.cols + kTile - 1) / kTile);
    case FP8BLK_DQF: return (n + dqf_chunk_elems<LPQ_DQF_U, LPQ_DQF_T>() - 1) / dqf_chunk_elems<LPQ_DQF_U, LPQ_DQF_T>();
    case MXFP8_Q:
    case MXFP8_QF: return (n + chunk_elems<LPQ_MXQ_U, LPQ_MXQ_T>() - 1) / chunk_elems<LPQ_MXQ_U, LPQ_MXQ_T>();
    case MXFP8_DQ: return (n + chunk_elems<LPQ_MXD_U, LPQ_MXD_T>() - 1) / chunk_elems<LPQ_MXD_U, LPQ_MXD_T>();
    case MXFP4_Q:
    case MXFP4_QF: return (n + chunk_elems<LPQ_MX4Q_U, LPQ_MX4Q_T>() - 1) / chunk_elems<LPQ_MX4Q_U, LPQ_MX4Q_T>();
    case MXFP4_DQ: return (n + chunk_elems<LPQ_MX4D_U, LPQ_MX4D_T>() - 1) / chunk_elems<LPQ_MX4D_U, LPQ_MX4D_T>();
    case MXFP4_QDQ:
    case MXFP4_QDQF: return (n + chunk_elems<LPQ_MX4QDQ_U, LPQ_MX4QDQ_T>() - 1) / chunk_elems<LPQ_MX4QDQ_U, LPQ_MX4QDQ_T>();
    case NV_AMAX: return (n + chunk_elems<LPQ_AMAX_U, LPQ_AMAX_T>() - 1) / chunk_elems<LPQ_AMAX_U, LPQ_AMAX_T>();
    case NV_Q: return (n + chunk_elems<LPQ_NVQ_U, LPQ_NVQ_T>() - 1) / chunk_elems<LPQ_NVQ_U, LPQ_NVQ_T>();
    case NV_DQ: return (n + chunk_elems<LPQ_NVD_U, LPQ_NVD_T>() - 1) / chunk_elems<LPQ_NVD_U, LPQ_NVD_T>();
    case NV_QDQ: return (n + chunk_elems<LPQ_QDQ_U, LPQ_QDQ_T>() - 1) / chunk_elems<LPQ_QDQ_U, LPQ_QDQ_T>();
    case NV_QDQ_W: return (n + chunk_elems<LPQ_QDQW_U, LPQ_QDQW_T>() - 1) / chunk_elems<LPQ_QDQW_U, LPQ_QDQW_T>();
    case I4_Q32:
    case I4_Q128: return (n + chunk_elems<LPQ_I4Q_U, LPQ_I4Q_T>() - 1) / chunk_elems<LPQ_I4Q_U, LPQ_I4Q_T>();
    case I4_DQ32:
    case I4_DQ128: return (n + chunk_elems<LPQ_I4D_U, LPQ_I4D_T>() - 1) / chunk_elems<LPQ_I4D_U, LPQ_I4D_T>();
    case I4_QDQ32:
    case I4_QDQ128: return (n + chunk_elems<LPQ_I4QDQ_U, LPQ_I4QDQ_T>() - 1) / chunk_elems<LPQ_I4QDQ_U, LPQ_I4QDQ_T>();
    default: return 0;
    }
}

int64_t units(Kind k, const lpq_requant_tensor& t) {
    const int64_t n = t.rows * t.cols;
    switch (k) {
    case RQ_FP8: return ((t.rows + kTile - 1) / kTile) * ((t.cols + kTile * LPQ_RQT_TW - 1) / (kTile * LPQ_RQT_TW));
    case RQ_MX: return (n + rq_chunk_elems<LPQ_RQM_U, LPQ_RQM_T>() - 1) / rq_chunk_elems<LPQ_RQM_U, LPQ_RQM_T>();
    case RQ_AMAX: return (n + rq_chunk_elems<LPQ_RQA_U, LPQ_RQA_T>() - 1) / rq_chunk_elems<LPQ_RQA_U, LPQ_RQA_T>();
    case RQ_NV: return (n + rq_chunk_elems<LPQ_RQN_U, LPQ_RQN_T>() - 1) / rq_chunk_elems<LPQ_RQN_U, LPQ_RQN_T>();
    default: return 0;
    }
}

// The most workgroups of a launch: the runtime takes fewer than 2^32 threads along a
// grid's axis, and the kernels' workgroup indexes are 32-bit.
constexpr int64_t max_groups(int threads) {
    const int64_t n = 0xffffffffLL / threads;
    return n < 0x7fffffffLL ? n : 0x7fffffffLL;
}

// Threads of a kind's workgroup, as dispatch() launches it.
int group_threads(Kind k) {
    switch (k) {
    case FP8BLK_Q: return 256 * LPQ_TILEQ_TW;
    case FP8BLK_QW: return 256 * LPQ_TILEQ_WIDE_TW;
    case FP8BLK_DQ: return LPQ_TILED_THREADS;
    case FP8BLK_DQF: return LPQ_DQF_T;
    case MXFP8_Q:
    case MXFP8_QF: return LPQ_MXQ_T;
    case MXFP8_DQ: return LPQ_MXD_T;
    case MXFP4_Q:
    case MXFP4_QF: return LPQ_MX4Q_T;
    case MXFP4_DQ: return LPQ_MX4D_T;
    case MXFP4_QDQ:
    case MXFP4_QDQF: return LPQ_MX4QDQ_T;
    case NV_AMAX: return LPQ_AMAX_T;
    case NV_Q: return LPQ_NVQ_T;
    case NV_DQ: return LPQ_NVD_T;
    case NV_QDQ: return LPQ_QDQ_T;
    case NV_QDQ_W: return LPQ_QDQW_T;
    case I4_Q32:
    case I4_Q128: return LPQ_I4Q_T;
    case I4_DQ32:
    case I4_DQ128: return LPQ_I4D_T;
    case I4_QDQ32:
    case I4_QDQ128: return LPQ_I4QDQ_T;
    case RQ_FP8: return 256 * LPQ_RQT_TW;
    case RQ_MX: return LPQ_RQM_T;
    case RQ_AMAX: return LPQ_RQA_T;
    case RQ_NV: return LPQ_RQN_T;
    }
    return 1024;
}

bool one_launch_holds(Kind k, int64_t units) { return units <= max_groups(group_threads(k)); }

void dispatch(Kind k, dim3 grid, hipStream_t stream, const lpq_tensor* tab, const lpq_tensor& one, const ChunkMap& map,
              const float* fa, float* fb) {
    const dim3 tileq(256 * LPQ_TILEQ_TW), tileqw(256 * LPQ_TILEQ_WIDE_TW), tiled(LPQ_TILED_THREADS);
    if (tab) {
        switch (k) {
        case FP8BLK_Q: hipLaunchKernelGGL((k_fp8blk_quant<LPQ_TILEQ_TW, true>), grid, tileq, 0, stream, tab, one, map); break;
        case FP8BLK_QW:
            hipLaunchKernelGGL((k_fp8blk_quant<LPQ_TILEQ_WIDE_TW, true>), grid, tileqw, 0, stream, tab, one, map);
            break;
        case FP8BLK_DQ: hipLaunchKernelGGL((k_fp8blk_dequant<LPQ_TILED_THREADS, true>), grid, tiled, 0, stream, tab, one, map); break;
        case FP8BLK_DQF: hipLaunchKernelGGL((k_fp8blk_dequant_flat<LPQ_DQF_U, LPQ_DQF_T, true>), grid, dim3(LPQ_DQF_T), 0, stream, tab, one, map); break;
        case MXFP8_Q: hipLaunchKernelGGL((k_mxfp8_quant<LPQ_MXQ_U, LPQ_MXQ_T, true>), grid, dim3(LPQ_MXQ_T), 0, stream, tab, one, map); break;
        case MXFP8_QF: hipLaunchKernelGGL((k_mxfp8_quant<LPQ_MXQ_U, LPQ_MXQ_T, true, true>), grid, dim3(LPQ_MXQ_T), 0, stream, tab, one, map); break;
        case MXFP8_DQ: hipLaunchKernelGGL((k_mxfp8_dequant<LPQ_MXD_U, LPQ_MXD_T, true>), grid, dim3(LPQ_MXD_T), 0, stream, tab, one, map); break;
        case MXFP4_Q: hipLaunchKernelGGL((k_mxfp4_quant<LPQ_MX4Q_U, LPQ_MX4Q_T, true>), grid, dim3(LPQ_MX4Q_T), 0, stream, tab, one, map); break;
        case MXFP4_QF: hipLaunchKernelGGL((k_mxfp4_quant<LPQ_MX4Q_U, LPQ_MX4Q_T, true, true>), grid, dim3(LPQ_MX4Q_T), 0, stream, tab, one, map); break;
        case MXFP4_DQ: hipLaunchKernelGGL((k_mxfp4_dequant<LPQ_MX4D_U, LPQ_MX4D_T, true>), grid, dim3(LPQ_MX4D_T), 0, stream, tab, one, map); break;
        case MXFP4_QDQ: hipLaunchKernelGGL((k_mxfp4_qdq<LPQ_MX4QDQ_U, LPQ_MX4QDQ_T, true>), grid, dim3(LPQ_MX4QDQ_T), 0, stream, tab, one, map); break;
        case MXFP4_QDQF: hipLaunchKernelGGL((k_mxfp4_qdq<LPQ_MX4QDQ_U, LPQ_MX4QDQ_T, true, true>), grid, dim3(LPQ_MX4QDQ_T), 0, stream, tab, one, map); break;
        case NV_AMAX: hipLaunchKernelGGL((k_amax<LPQ_AMAX_U, LPQ_AMAX_T, true>), grid, dim3(LPQ_AMAX_T), 0, stream, tab, one, map, fb); break;
        case NV_Q: hipLaunchKernelGGL((k_nvfp4_quant<LPQ_NVQ_U, LPQ_NVQ_T, true>), grid, dim3(LPQ_NVQ_T), 0, stream, tab, one, map, fa, fb); break;
        case NV_DQ: hipLaunchKernelGGL((k_nvfp4_dequant<LPQ_NVD_U, LPQ_NVD_T, true>), grid, dim3(LPQ_NVD_T), 0, stream, tab, one, map, fa); break;
        case NV_QDQ: hipLaunchKernelGGL((k_nvfp4_qdq<LPQ_QDQ_U, LPQ_QDQ_T, true>), grid, dim3(LPQ_QDQ_T), 0, stream, tab, one, map, fa); break;
        case I4_Q32: hipLaunchKernelGGL((k_int4_quant<LPQ_I4Q_U, LPQ_I4Q_T, true, 32>), grid, dim3(LPQ_I4Q_T), 0, stream, tab, one, map); break;
        case I4_Q128: hipLaunchKernelGGL((k_int4_quant<LPQ_I4Q_U, LPQ_I4Q_T, true, 128>), grid, dim3(LPQ_I4Q_T), 0, stream, tab, one, map); break;
        case I4_DQ32: hipLaunchKernelGGL((k_int4_dequant<LPQ_I4D_U, LPQ_I4D_T, true, 32>), grid, dim3(LPQ_I4D_T), 0, stream, tab, one, map); break;
        case I4_DQ128: hipLaunchKernelGGL((k_int4_dequant<LPQ_I4D_U, LPQ_I4D_T, true, 128>), grid, dim3(LPQ_I4D_T), 0, stream, tab, one, map); break;
        case I4_QDQ32: hipLaunchKernelGGL((k_int4_qdq<LPQ_I4QDQ_U, LPQ_I4QDQ_T, true, 32>), grid, dim3(LPQ_I4QDQ_T), 0, stream, tab, one, map); break;
        case I4_QDQ128: hipLaunchKernelGGL((k_int4_qdq<LPQ_I4QDQ_U, LPQ_I4QDQ_T, true, 128>), grid, dim3(LPQ_I4QDQ_T), 0, stream, tab, one, map); break;
        default: break;
        }
    } else {
        switch (k) {
        case FP8BLK_Q: hipLaunchKernelGGL((k_fp8blk_quant<LPQ_TILEQ_TW, false>), grid, tileq, 0, stream, tab, one, map); break;
        case FP8BLK_QW:
            hipLaunchKernelGGL((k_fp8blk_quant<LPQ_TILEQ_WIDE_TW, false>), grid, tileqw, 0, stream, tab, one, map);
            break;
        case FP8BLK_DQ: hipLaunchKernelGGL((k_fp8blk_dequant<LPQ_TILED_THREADS, false>), grid, tiled, 0, stream, tab, one, map); break;
        case FP8BLK_DQF: hipLaunchKernelGGL((k_fp8blk_dequant_flat<LPQ_DQF_U, LPQ_DQF_T, false>), grid, dim3(LPQ_DQF_T), 0, stream, tab, one, map); break;
        case MXFP8_Q: hipLaunchKernelGGL((k_mxfp8_quant<LPQ_MXQ_U, LPQ_MXQ_T, false>), grid, dim3(LPQ_MXQ_T), 0, stream, tab, one, map); break;
        case MXFP8_QF: hipLaunchKernelGGL((k_mxfp8_quant<LPQ_MXQ_U, LPQ_MXQ_T, false, true>), grid, dim3(LPQ_MXQ_T), 0, stream, tab, one, map); break;
        case MXFP8_DQ: hipLaunchKernelGGL((k_mxfp8_dequant<LPQ_MXD_U, LPQ_MXD_T, false>), grid, dim3(LPQ_MXD_T), 0, stream, tab, one, map); break;
        case MXFP4_Q: hipLaunchKernelGGL((k_mxfp4_quant<LPQ_MX4Q_U, LPQ_MX4Q_T, false>), grid, dim3(LPQ_MX4Q_T), 0, stream, tab, one, map); break;
        case MXFP4_QF: hipLaunchKernelGGL((k_mxfp4_quant<LPQ_MX4Q_U, LPQ_MX4Q_T, false, true>), grid, dim3(LPQ_MX4Q_T), 0, stream, tab, one, map); break;
        case MXFP4_DQ: hipLaunchKernelGGL((k_mxfp4_dequant<LPQ_MX4D_U, LPQ_MX4D_T, false>), grid, dim3(LPQ_MX4D_T), 0, stream, tab, one, map); break;
        case MXFP4_QDQ: hipLaunchKernelGGL((k_mxfp4_qdq<LPQ_MX4QDQ_U, LPQ_MX4QDQ_T, false>), grid, dim3(LPQ_MX4QDQ_T), 0, stream, tab, one, map); break;
        case MXFP4_QDQF: hipLaunchKernelGGL((k_mxfp4_qdq<LPQ_MX4QDQ_U, LPQ_MX4QDQ_T, false, true>), grid, dim3(LPQ_MX4QDQ_T), 0, stream, tab, one, map); break;
        case NV_AMAX: hipLaunchKernelGGL((k_amax<LPQ_AMAX_U, LPQ_AMAX_T, false>), grid, dim3(LPQ_AMAX_T), 0, stream, tab, one, map, fb); break;
        case NV_Q: hipLaunchKernelGGL((k_nvfp4_quant<LPQ_NVQ_U, LPQ_NVQ_T, false>), grid, dim3(LPQ_NVQ_T), 0, stream, tab, one, map, fa, fb); break;
        case NV_DQ: hipLaunchKernelGGL((k_nvfp4_dequant<LPQ_NVD_U, LPQ_NVD_T, false>), grid, dim3(LPQ_NVD_T), 0, stream, tab, one, map, fa); break;
        case NV_QDQ: hipLaunchKernelGGL((k_nvfp4_qdq<LPQ_QDQ_U, LPQ_QDQ_T, false>), grid, dim3(LPQ_QDQ_T), 0, stream, tab, one, map, fa); break;
        case NV_QDQ_W:
            hipLaunchKernelGGL((k_nvfp4_qdq<LPQ_QDQW_U, LPQ_QDQW_T, false, LPQ_QDQW_AHEAD != 0>), grid, dim3(LPQ_QDQW_T), 0,
                               stream, tab, one, map, fa);
            break;
        case I4_Q32: hipLaunchKernelGGL((k_int4_quant<LPQ_I4Q_U, LPQ_I4Q_T, false, 32>), grid, dim3(LPQ_I4Q_T), 0, stream, tab, one, map); break;
        case I4_Q128: hipLaunchKernelGGL((k_int4_quant<LPQ_I4Q_U, LPQ_I4Q_T, false, 128>), grid, dim3(LPQ_I4Q_T), 0, stream, tab, one, map); break;
        case I4_DQ32: hipLaunchKernelGGL((k_int4_dequant<LPQ_I4D_U, LPQ_I4D_T, false, 32>), grid, dim3(LPQ_I4D_T), 0, stream, tab, one, map); break;
        case I4_DQ128: hipLaunchKernelGGL((k_int4_dequant<LPQ_I4D_U, LPQ_I4D_T, false, 128>), grid, dim3(LPQ_I4D_T), 0, stream, tab, one, map); break;
        case I4_QDQ32: hipLaunchKernelGGL((k_int4_qdq<LPQ_I4QDQ_U, LPQ_I4QDQ_T, false, 32>), grid, dim3(LPQ_I4QDQ_T), 0, stream, tab, one, map); break;
        case I4_QDQ128: hipLaunchKernelGGL((k_int4_qdq<LPQ_I4QDQ_U, LPQ_I4QDQ_T, false, 128>), grid, dim3(LPQ_I4QDQ_T), 0, stream, tab, one, map); break;
        default: break;
        }
    }
}

void dispatch(Kind k, dim3 grid, hipStream_t stream, const lpq_requant_tensor* tab, const lpq_requant_tensor& one,
              const ChunkMap& map, const float* fa, float* fb) {
    const dim3 tile(256 * LPQ_RQT_TW);
    if (tab) {
        switch (k) {
        case RQ_FP8: hipLaunchKernelGGL((k_requant_fp8blk<LPQ_RQT_TW, true>), grid, tile, 0, stream, tab, one, map); break;
        case RQ_MX: hipLaunchKernelGGL((k_requant_mxfp8<LPQ_RQM_U, LPQ_RQM_T, true>), grid, dim3(LPQ_RQM_T), 0, stream, tab, one, map); break;
        case RQ_AMAX: hipLaunchKernelGGL((k_requant_amax<LPQ_RQA_U, LPQ_RQA_T, true>), grid, dim3(LPQ_RQA_T), 0, stream, tab, one, map, fb); break;
        case RQ_NV: hipLaunchKernelGGL((k_requant_nvfp4<LPQ_RQN_U, LPQ_RQN_T, true>), grid, dim3(LPQ_RQN_T), 0, stream, tab, one, map, fa, fb); break;
        default: break;
        }
    } else {
        switch (k) {
        case RQ_FP8: hipLaunchKernelGGL((k_requant_fp8blk<LPQ_RQT_TW, false>), grid, tile, 0, stream, tab, one, map); break;
        case RQ_MX: hipLaunchKernelGGL((k_requant_mxfp8<LPQ_RQM_U, LPQ_RQM_T, false>), grid, dim3(LPQ_RQM_T), 0, stream, tab, one, map); break;
        case RQ_AMAX: hipLaunchKernelGGL((k_requant_amax<LPQ_RQA_U, LPQ_RQA_T, false>), grid, dim3(LPQ_RQA_T), 0, stream, tab, one, map, fb); break;
        case RQ_NV: hipLaunchKernelGGL((k_requant_nvfp4<LPQ_RQN_U, LPQ_RQN_T, false>), grid, dim3(LPQ_RQN_T), 0, stream, tab, one, map, fa, fb); break;
        default: break;
        }
    }
}

// Where the launch over tensors [i0, count) stops: the first tensor that would
// exceed kMaxSeg segments (runs of equal work-unit counts) or max_groups work units.
// Fills map and total; returns -1 when one tensor alone is too large.
template <typename D>
int32_t slice_end(Kind k, const D* host, int32_t count, int32_t i0, const D& one, ChunkMap& map, int64_t& total) {
    map = ChunkMap{};
    total = 0;
    const int64_t most = max_groups(group_threads(k));
    int32_t nseg = 0, i = i0;
    while (i < count) {
        const int64_t u = units(k, host ? host[i] : one);
        if (u > most) return -1;
        if (total + u > most) break;
        if (nseg == 0 || (int64_t)map.units[nseg - 1] != u) {
            if (nseg == kMaxSeg) break;
            map.first[nseg] = (uint32_t)total;
            map.tensor0[nseg] = (uint32_t)(i - i0);
            map.units[nseg] = (uint32_t)u;
            map.inv_units[nseg] = 1.0 / (double)u;
            nseg++;
        }
        total += u;
        i++;
    }
    map.nseg = nseg;
    return i;
}

// Number of launches a call of kind k over host[0, n) takes (-1: a tensor is too large).
template <typename D>
int64_t launch_count(Kind k, const D* host, int32_t n) {
    int64_t launches = 0;
    ChunkMap map;
    int64_t total;
    for (int32_t i0 = 0; i0 < n; launches++) {
        const int32_t i = slice_end(k, host, n, i0, D{}, map, total);
        if (i < 0) return -1;
        i0 = i;
    }
    return launches;
}

// Launch kernel `k` over tensors [0, n) of `host`/`dev` (single tensor: dev ==
// nullptr, `one` used), in slices of at most kMaxSeg segments and max_groups work
// units.
template <typename D>
lpq_status launch(Kind k, const D* host, const D* dev, int32_t n, const D& one, const float* fa, float* fb,
                  hipStream_t stream, float gdiv = 2688.0f) {
    const int32_t count = dev ? n : 1;
    int32_t i0 = 0;
    while (i0 < count) {
        ChunkMap map;
        int64_t total;
        const int32_t i = slice_end(k, dev ? host : nullptr, count, i0, one, map, total);
        if (i < 0) return LPQ_ERR_SHAPE;
        map.gdiv = gdiv;
        dispatch(k, dim3((unsigned)total), stream, dev ? dev + i0 : nullptr, one, map, fa, fb);
        lpq_status st = launched();
        if (st != LPQ_OK) return st;
        i0 = i;
    }
    return LPQ_OK;
}

lpq_tensor make_one(const void* src, void* dst, void* scale, int64_t M, int64_t N) {
    lpq_tensor t;
    t.src = src;
    t.dst = dst;
    t.scale = scale;
    t.rows = M;
    t.cols = N;
    t.group = 0;
    t.reserved = 0;
    return t;
}

template <typename D>
lpq_status single(Kind k, const D& one, const float* fa, float* fb, void* stream, float gdiv = 2688.0f) {
    lpq_status st = check_tensor(k, one, 0);
    if (st != LPQ_OK) return st;
    return launch<D>(k, nullptr, nullptr, 0, one, fa, fb, (hipStream_t)stream, gdiv);
}

// Checks of a grouped call's tables and of every descriptor for kind k.
template <typename D>
lpq_status check_grouped(Kind k, const D* host, const D* dev, int32_t n, int32_t n_groups) {
    if (!host || !dev) return LPQ_ERR_NULL;
    if (n <= 0) return LPQ_ERR_SHAPE;
    if (!aligned(dev, 8)) return LPQ_ERR_ALIGN;
    for (int32_t i = 0; i < n; i++) {
        lpq_status st = check_tensor(k, host[i], n_groups);
        if (st != LPQ_OK) return st;
    }
    return LPQ_OK;
}

template <typename D>
lpq_status grouped(Kind k, const D* host, const D* dev, int32_t n, int32_t n_groups, const float* fa, float* fb,
                   void* stream, float gdiv = 2688.0f) {
    lpq_status st = check_grouped(k, host, dev, n, n_groups);
    if (st != LPQ_OK) return st;
    return launch<D>(k, host, dev, n, D{}, fa, fb, (hipStream_t)stream, gdiv);
}

// Strip width of a block-FP8 quantize call: 4 tiles per workgroup when the
// call has at least LPQ_TILEQ_WIDE_MIN 4-tile strips and takes no more
// launches that way, else LPQ_TILEQ_TW.  Measured: wide strips run faster on
// large launches (longer contiguous row runs) and slower on short ones, where
// fewer, longer workgroups leave more of the chip idle at the end.  The launch
// count matters when the table alternates shapes: Qwen3-30B-A3B experts
// (768x2048, 2048x768) have equal 2-tile strip counts, one run of equal work
// units, but unequal 4-tile counts, a new run at every tensor.  Any tensor that
// fails the checks keeps the narrow kind (the call is refused later).
Kind fp8blk_quant_kind(const lpq_tensor* t, int32_t n) {
    if (!t || n <= 0) return FP8BLK_Q;
    int64_t strips = 0;
    for (int32_t i = 0; i < n; i++) {
        if (check_tensor(FP8BLK_QW, t[i], 0) != LPQ_OK) return FP8BLK_Q;
        strips += units(FP8BLK_QW, t[i]);
    }
    if (strips < LPQ_TILEQ_WIDE_MIN) return FP8BLK_Q;
    const int64_t wide = launch_count(FP8BLK_QW, t, n), narrow = launch_count(FP8BLK_Q, t, n);
    return wide > 0 && wide <= narrow ? FP8BLK_QW : FP8BLK_Q;
}

// The kind of an INT4 operation ("INT4 QAT 训练") for a group size of 32 or
// 128; -1 for any other group size (the call returns LPQ_ERR_ARG).
int int4_kind(Kind k32, Kind k128, int32_t group) { return group == 32 ? k32 : group == 128 ? k128 : -1; }

// 6 * the E4M3 maximum of an NVFP4 call, or 0 for an unsupported maximum.
float gdiv_of(int e4m3_max) { return e4m3_max == 448 ? 2688.0f : (e4m3_max == 256 ? 1536.0f : 0.0f); }

lpq_requant_tensor make_requant(const uint8_t* q, const float* s, void* dst, void* dst_scale, int64_t M, int64_t N) {
    lpq_requant_tensor t;
    t.src = q;
    t.src_scale = s;
    t.dst = dst;
    t.dst_scale = dst_scale;
    t.rows = M;
    t.cols = N;
    t.group = 0;
    t.reserved = 0;
    return t;
}

lpq_status fill(float* p, int64_t n, float v, void* stream) {
    hipLaunchKernelGGL(k_fill_f32, dim3((unsigned)((n + kThreads - 1) / kThreads)), dim3(kThreads), 0,
                       (hipStream_t)stream, p, n, v);
    return launched();
}

lpq_status global_scale(const float* amax, int32_t n, float* out, float gdiv, void* stream) {
    hipLaunchKernelGGL(k_global_scale, dim3((unsigned)((n + kThreads - 1) / kThreads)), dim3(kThreads), 0,
                       (hipStream_t)stream, amax, n, out, gdiv);
    return launched();
}

// The single-tensor QDQ kind for n elements: a tensor of at most a few waves
// of full-CU workgroups takes the wide shape (every load of a lane issued up
// front); larger ones stream.
Kind qdq_kind(int64_t n) { return n <= LPQ_QDQW_MAX_ELEMS ? NV_QDQ_W : NV_QDQ; }

// NVFP4 quantize (k = NV_Q) or QDQ (k = NV_QDQ) of one tensor.  With amax ==
// NULL the tensor's own amax is the group amax ("verl NVFP4 QAT" 2.3: a tensor
// of its own is a group of one), computed by the call into a word the caller
// already owns, and every launch goes on the caller's stream, so each sees the
// previous one's result:
//   quantize: the g word is cleared, receives max |w| from the amax pass, is
//     read as A by the encode (which then leaves it alone), and is finally
//     turned into fl(A / gdiv);
//   QDQ: the first word of y is cleared and receives max |x|; the QDQ of every
//     element but the first 16-element block reads A from it; the QDQ of that
//     block runs last, reading A before it writes the block over the word
//     (only its first wave holds elements, and each lane reads A before its
//     store).  x and y must not overlap.
lpq_status nvfp4_single(Kind k, const uint16_t* w, int64_t M, int64_t N, const float* amax, int e4m3_max, void* dst,
                        void* scale, float* g, void* stream) {
    if (k == NV_Q && !g) return LPQ_ERR_NULL;
    if ((amax && !aligned(amax, 4)) || (g && !aligned(g, 4))) return LPQ_ERR_ALIGN;
    const float gdiv = gdiv_of(e4m3_max);
    if (gdiv == 0.0f) return LPQ_ERR_ARG;
    const lpq_tensor one = make_one(w, dst, scale, M, N);
    lpq_status st = check_tensor(k, one, 0);
    if (st != LPQ_OK) return st;
    const hipStream_t s = (hipStream_t)stream;
    const int64_t n = M * N;
    if (amax) {
        const Kind kk = k == NV_QDQ ? qdq_kind(n) : k;
        return launch<lpq_tensor>(kk, nullptr, nullptr, 0, one, amax, k == NV_Q ? g : nullptr, s, gdiv);
    }
    if (k == NV_Q) {
        if ((st = fill(g, 1, 0.0f, stream)) != LPQ_OK) return st;
        if ((st = launch<lpq_tensor>(NV_AMAX, nullptr, nullptr, 0, one, nullptr, g, s)) != LPQ_OK) return st;
        if ((st = launch<lpq_tensor>(NV_Q, nullptr, nullptr, 0, one, g, nullptr, s, gdiv)) != LPQ_OK) return st;
        return global_scale(g, 1, g, gdiv, stream);
    }
    uint16_t* y = static_cast<uint16_t*>(dst);
    const uintptr_t xa = reinterpret_cast<uintptr_t>(w), ya = reinterpret_cast<uintptr_t>(y);
    if (xa < ya + 2 * (uint64_t)n && ya < xa + 2 * (uint64_t)n) return LPQ_ERR_ARG;   // overlapping x and y
    float* a = reinterpret_cast<float*>(y);
    if ((st = fill(a, 1, 0.0f, stream)) != LPQ_OK) return st;
    if ((st = launch<lpq_tensor>(NV_AMAX, nullptr, nullptr, 0, one, nullptr, a, s)) != LPQ_OK) return st;
    if (n > 16) {
        const lpq_tensor tail = make_one(w + 16, y + 16, nullptr, 1, n - 16);
        if ((st = launch<lpq_tensor>(qdq_kind(n - 16), nullptr, nullptr, 0, tail, a, nullptr, s, gdiv)) != LPQ_OK)
            return st;
    }
    const lpq_tensor head = make_one(w, y, nullptr, 1, 16);
    return launch<lpq_tensor>(NV_QDQ_W, nullptr, nullptr, 0, head, a, nullptr, s, gdiv);
}

// Grouped NVFP4 quantize (NV_Q) or QDQ (NV_QDQ).  amax_valid != 0: group_amax
// holds each group's A (a cached or observed value, or lpq_nvfp4_amax_grouped's
// result) and is only read.  amax_valid == 0: the call fills it first -- the
// slots are cleared and the amax pass folds every member's max |w| into its
// group's slot (the group maximum, "verl NVFP4 QAT" 2.4) -- then encodes.
lpq_status nvfp4_grouped(Kind k, const lpq_tensor* host, const lpq_tensor* dev, int32_t n, float* group_amax,
                         int32_t n_groups, int amax_valid, int e4m3_max, float* group_g, void* stream) {
    if (!group_amax || (k == NV_Q && !group_g)) return LPQ_ERR_NULL;
    if (n_groups <= 0) return LPQ_ERR_SHAPE;
    if (!aligned(group_amax, 4) || (group_g && !aligned(group_g, 4))) return LPQ_ERR_ALIGN;
    const float gdiv = gdiv_of(e4m3_max);
    if (gdiv == 0.0f) return LPQ_ERR_ARG;
    lpq_status st = check_grouped(k, host, dev, n, n_groups);   // every amax-pass condition included
    if (st != LPQ_OK) return st;
    const hipStream_t s = (hipStream_t)stream;
    if (!amax_valid) {
        if ((st = fill(group_amax, n_groups, 0.0f, stream)) != LPQ_OK) return st;
        if ((st = launch<lpq_tensor>(NV_AMAX, host, dev, n, lpq_tensor{}, nullptr, group_amax, s)) != LPQ_OK) return st;
    }
    return launch<lpq_tensor>(k, host, dev, n, lpq_tensor{}, group_amax, k == NV_Q ? group_g : nullptr, s, gdiv);
}

// Two byte ranges that share a byte (either may be empty).
inline bool overlap(const void* a, int64_t na, const void* b, int64_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return na > 0 && nb > 0 && x < y + (uintptr_t)nb && y < x + (uintptr_t)na;
}

template <bool FP4>
lpq_status mx_transpose(const uint16_t* w, int64_t M, int64_t N, int floor_rule, uint8_t* q, uint8_t* e, uint8_t* qt,
                        uint8_t* et, void* stream) {
    if (M <= 0 || N <= 0 || N % 32 || M > (int64_t(1) << 40) / N) return LPQ_ERR_SHAPE;
    if (!w || !qt || !et || !q != !e) return LPQ_ERR_NULL;
    if (floor_rule != 0 && floor_rule != 1) return LPQ_ERR_ARG;
    if (!aligned(w, 16) || !aligned(qt, 16) || (q && !aligned(q, FP4 ? 4 : 8))) return LPQ_ERR_ALIGN;
    TransposeArgs A;
    A.w = w;
    A.q = q;
    A.e = e;
    A.qt = qt;
    A.et = et;
    A.M = M;
    A.N = N;
    A.Mp = (M + 31) / 32 * 32;
    A.tiles_n = (N + kTrN - 1) / kTrN;
    const int64_t code = FP4 ? 2 : 1;   // codes in a byte
    const struct { const void* p; int64_t n; } out[] = {
        {qt, N * A.Mp / code}, {et, N * A.Mp / 32}, {q, q ? M * N / code : 0}, {e, e ? M * N / 32 : 0}};
    for (int i = 0; i < 4; i++) {
        if (overlap(w, 2 * M * N, out[i].p, out[i].n)) return LPQ_ERR_ARG;
        for (int j = 0; j < i; j++)
            if (overlap(out[i].p, out[i].n, out[j].p, out[j].n)) return LPQ_ERR_ARG;
    }
    const int64_t tiles = (M + kTrM - 1) / kTrM * A.tiles_n, most = max_groups(kTrThreads);
    const dim3 block(kTrThreads);
    const hipStream_t s = (hipStream_t)stream;
    for (A.first = 0; A.first < tiles; A.first += most) {
        const dim3 grid((unsigned)(tiles - A.first < most ? tiles - A.first : most));
        if (floor_rule) {
            if (q) hipLaunchKernelGGL((k_mx_transpose<FP4, true, true>), grid, block, 0, s, A);
            else hipLaunchKernelGGL((k_mx_transpose<FP4, true, false>), grid, block, 0, s, A);
        } else {
            if (q) hipLaunchKernelGGL((k_mx_transpose<FP4, false, true>), grid, block, 0, s, A);
            else hipLaunchKernelGGL((k_mx_transpose<FP4, false, false>), grid, block, 0, s, A);
        }
        const lpq_status st = launched();
        if (st != LPQ_OK) return st;
    }
    return LPQ_OK;
}

// Shape of a norm call: whole MXFP8 blocks, a row that fits the kernels' registers.
lpq_status norm_shape(int64_t M, int64_t N) {
    if (M <= 0 || N <= 0 || N % 32 || N > kNormMaxN || M > (int64_t(1) << 40) / N) return LPQ_ERR_SHAPE;
    return LPQ_OK;
}

lpq_status rmsnorm(const NormArgs& A, void* stream) {
    lpq_status st = norm_shape(A.M, A.N);
    if (st != LPQ_OK) return st;
    if (!A.x || !A.gamma || (!A.y && !A.q) || !A.q != !A.e || (A.residual && !A.h)) return LPQ_ERR_NULL;
    if (!A.residual && A.h) return LPQ_ERR_ARG;   // without a residual h is x
    if (!(A.eps > 0.0f) || A.eps > 3.4028235e38f) return LPQ_ERR_ARG;
    if (!aligned(A.x, 16) || !aligned(A.residual, 16) || !aligned(A.gamma, 16) || !aligned(A.h, 16) || !aligned(A.y, 16) ||
        !aligned(A.q, 8) || !aligned(A.rstd, 4))
        return LPQ_ERR_ALIGN;
    const int64_t n = A.M * A.N;
    const struct { const void* p; int64_t n; } in[] = {{A.x, 2 * n}, {A.residual, A.residual ? 2 * n : 0}, {A.gamma, 2 * (int64_t)A.N}},
        out[] = {{A.h, A.h ? 2 * n : 0}, {A.y, A.y ? 2 * n : 0}, {A.q, A.q ? n : 0}, {A.e, A.e ? n / 32 : 0}, {A.rstd, A.rstd ? 4 * A.M : 0}};
    for (int i = 0; i < 5; i++) {
        for (int j = 0; j < 3; j++)   // h may be x or the residual itself: a lane reads what it writes first
            if (!(i == 0 && j < 2 && in[j].p == out[i].p) && overlap(out[i].p, out[i].n, in[j].p, in[j].n)) return LPQ_ERR_ARG;
        for (int j = 0; j < i; j++)
            if (overlap(out[i].p, out[i].n, out[j].p, out[j].n)) return LPQ_ERR_ARG;
    }
    return by_row(A.N, [&](auto shape) {
        constexpr int G = decltype(shape)::g, U = decltype(shape)::u, kRows = norm_threads(G) / G;
        constexpr int64_t most = max_groups(norm_threads(G)) * kRows;   // rows of a launch
        for (int64_t row = 0; row < A.M; row += most) {
            NormArgs S = A;
            const int64_t at = row * A.N;
            S.x += at;
            if (S.residual) S.residual += at;
            if (S.h) S.h += at;
            if (S.y) S.y += at;
            if (S.rstd) S.rstd += row;
            if (S.q) S.q += at;
            if (S.e) S.e += at / 32;
            S.M = A.M - row < most ? A.M - row : most;
            hipLaunchKernelGGL((k_rmsnorm<G, U>), dim3((unsigned)((S.M + kRows - 1) / kRows)), dim3(norm_threads(G)), 0,
                               (hipStream_t)stream, S);
            const lpq_status st = launched();
            if (st != LPQ_OK) return st;
        }
        return LPQ_OK;
    });
}

// Workgroups of the backward pass, each with a partial sum of dgamma that costs
// 8 bytes a column: one per CU for long rows (8192 x 2560: 34 us with 256, 38
// with 512, 44 with 1024), up to four for short ones, whose partial sums are
// small and whose loads need more waves to wait beside (98301 x 128: 29, 18 and
// 15 us).
int64_t norm_grad_groups(int64_t M, int64_t N) {
    return by_row(N, [&](auto shape) {
        constexpr int G = decltype(shape)::g, kRows = norm_threads(G) / G;
        const int64_t groups = (M + kRows - 1) / kRows, each = 1024 / N, most = kComputeUnits * (each < 1 ? 1 : each > 4 ? 4 : each);
        return groups < most ? groups : most;
    });
}

lpq_status rmsnorm_grad(NormGradArgs A, float* dgamma, int accumulate, void* workspace, int64_t workspace_bytes, void* stream) {
    lpq_status st = norm_shape(A.M, A.N);
    if (st != LPQ_OK) return st;
    if (!A.dy || !A.h || !A.gamma || !A.rstd || !A.dx || (dgamma && !workspace)) return LPQ_ERR_NULL;
    if (!aligned(A.dy, 16) || !aligned(A.h, 16) || !aligned(A.gamma, 16) || !aligned(A.dres, 16) || !aligned(A.dx, 16) ||
        !aligned(A.rstd, 4) || !aligned(dgamma, 4) || !aligned(workspace, 16))
        return LPQ_ERR_ALIGN;
    const int64_t n = A.M * A.N, groups = norm_grad_groups(A.M, A.N), need = dgamma ? 4 * groups * A.N : 0;
    if (workspace_bytes < need) return LPQ_ERR_ARG;
    const struct { const void* p; int64_t n; } in[] = {{A.dy, 2 * n}, {A.dres, A.dres ? 2 * n : 0}, {A.h, 2 * n},
                                                       {A.gamma, 2 * (int64_t)A.N}, {A.rstd, 4 * A.M}},
        out[] = {{A.dx, 2 * n}, {dgamma, dgamma ? 4 * (int64_t)A.N : 0}, {workspace, need}};
    for (int i = 0; i < 3; i++) {
        for (int j = 0; j < 5; j++)   // dx may be dy or dres itself
            if (!(i == 0 && j < 2 && in[j].p == out[i].p) && overlap(out[i].p, out[i].n, in[j].p, in[j].n)) return LPQ_ERR_ARG;
        for (int j = 0; j < i; j++)
            if (overlap(out[i].p, out[i].n, out[j].p, out[j].n)) return LPQ_ERR_ARG;
    }
    A.part = dgamma ? static_cast<float*>(workspace) : nullptr;
    const hipStream_t s = (hipStream_t)stream;
    st = by_row(A.N, [&](auto shape) {
        constexpr int G = decltype(shape)::g, U = decltype(shape)::u;
        hipLaunchKernelGGL((k_rmsnorm_grad<G, U>), dim3((unsigned)groups), dim3(norm_threads(G)), 0, s, A);
        return launched();
    });
    if (st != LPQ_OK || !dgamma) return st;
    hipLaunchKernelGGL(k_rmsnorm_dgamma, dim3((unsigned)((A.N + kDgCols - 1) / kDgCols)), dim3(kDgCols * kDgSlices), 0, s, A.part,
                       (int32_t)groups, A.N, accumulate, dgamma);
    return launched();
}

template <int N>
using Int = std::integral_constant<int, N>;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Which kernel a product takes.  Both sides were timed for the four format pairs
// at k = 2560 and 9728; times here are us of MXFP8 / MXFP8 x MXFP4 / MXFP4.
//  * Tiles of 128 x 128 or more by way of LDS, from 128 rows and 64 such tiles on:
//    fewer leave most of the card idle, and a stage's way from memory to LDS takes as
//    long for one tile as for 256.  128 x 9728 x 2560 (76 tiles): 18 / 17 / 12 in
//    tiles, 28 / 24 / 19 by rows; 512 x 2560 x 9728 (80): 57 / 55 / 37 and 89 / 72 /
//    56.  256 x 2560 (40): 18 / 17 / 12 in tiles, 15 / 13 / 11 by rows at k = 2560; 57 /
//    55 / 37 and 46 / 37 / 29 at 9728.  A tile has 128 rows to itself, so 65 to 127
//    rows go by rows where tiles might be faster: 127 x 9728 x 2560 takes 28 / 24 / 19.
//  * Among the tiles the shape that takes the least time for its rounds of the
//    card.  One round (256 tiles, one on each CU) of 256 x 256 counts 2; 256 x 192
//    1.8; 128 x 128 0.95 alone, 1.1 with two on each CU, and 1.6 where many rounds
//    keep memory busy, which larger tiles ask less of.  These are MXFP8's times at k =
//    2560 (37 us, 33 us, 16 and 20 us, 28 us a round) and decide the other pairs and k
//    too: of 14 sizes from 1024 x 2560 x 2560 to 8192 x 8192 x 8192 the choice is within
//    10% of the fastest shape at 12; 2048 x 9728 x 9728 takes 256 / 210 / 155 by 128 x
//    128 and 225 / 196 / 133 by 256 x 192, 8192 x 8192 x 512 52 / 49 / 41 by 256 x 256
//    and 48 / 46 / 37 by 256 x 192.
//  * Rows otherwise, in workgroups of as many rows of b as leave 128 workgroups: each
//    reads its rows of a once (64 x 9728 x 2560: 23 us with 16, 19 with 32 and 14
//    with 64; 64 x 2560 x 2560, 40 workgroups with 64: 9 us with 16, 12 with 64).
template <bool FP4A, bool FP4B>
lpq_status mx_matmul(const MatmulArgs& A, hipStream_t s) {
    auto rows = [&](auto nt, auto mt, auto u) {
        constexpr int NT = decltype(nt)::value, MT = decltype(mt)::value, U = decltype(u)::value;
        const int64_t tiles_n = ceil_div(A.N, 16 * NT), tiles = ceil_div(A.M, 16 * MT) * tiles_n, most = max_groups(64 * kRowsWaves);
        if (tiles > 0x7fffffffLL) return LPQ_ERR_SHAPE;   // tile indexes are 32-bit
        for (int64_t first = 0; first < tiles; first += most) {
            hipLaunchKernelGGL((k_mx_matmul_rows<FP4B, FP4A, NT, MT, U>), dim3((unsigned)(tiles - first < most ? tiles - first : most)),
                               dim3(64 * kRowsWaves), 0, s, A, (int)tiles_n, (int)first);
            const lpq_status st = launched();
            if (st != LPQ_OK) return st;
        }
        return LPQ_OK;
    };
    auto tile = [&](auto tn, auto tm, auto wn, auto wm) {
        constexpr int TN = decltype(tn)::value, TM = decltype(tm)::value, WN = decltype(wn)::value, WM = decltype(wm)::value;
        const int64_t nt = ceil_div(A.N, TN), mt = ceil_div(A.M, TM);
        if (nt * mt > 0x7fffffffLL) return LPQ_ERR_SHAPE;   // tile indexes are 32-bit
        const int64_t most = kComputeUnits * (TN == 256 ? 1 : 2);   // as many as run at one time: they go on from tile to tile
        hipLaunchKernelGGL((k_mx_matmul_tile<FP4B, FP4A, TN, TM, WN, WM>), dim3((unsigned)(nt * mt < most ? nt * mt : most)),
                           dim3(64 * WN * WM), 0, s, A, (int)nt, (int)mt);
        return launched();
    };
    const int64_t n128 = ceil_div(A.N, 128) * ceil_div(A.M, 128);
    const bool limits = A.K > 128 * stage_steps<FP4B, FP4A>() && A.K <= (1 << 22) && A.N <= (1 << 22);
    if (limits && A.M >= 128 && A.N >= 128 && n128 >= 64) {
        const double none = 1e30;
        const double c128 = n128 <= 256 ? 0.95 : ceil_div(n128, 512) * (n128 <= 2048 ? 1.1 : 1.6);
        const double c256 = A.M >= 256 && A.N >= 256 ? 2.0 * ceil_div(ceil_div(A.N, 256) * ceil_div(A.M, 256), 256) : none;
        if constexpr (!FP4A || FP4B) {   // an E2M1 a beside an E4M3 b has too few pieces for 192 rows
            const double c192 = A.M >= 192 && A.N >= 256 ? 1.8 * ceil_div(ceil_div(A.N, 256) * ceil_div(A.M, 192), 256) : none;
            if (c192 < c256 && c192 < c128) return tile(Int<256>{}, Int<192>{}, Int<2>{}, Int<4>{});
        }
        if (c256 < c128) return tile(Int<256>{}, Int<256>{}, Int<2>{}, Int<4>{});
        return tile(Int<128>{}, Int<128>{}, Int<2>{}, Int<2>{});
    }
    if (A.M <= 16) return rows(Int<1>{}, Int<1>{}, Int<3>{});
    const int64_t mt = A.M <= 32 ? 1 : ceil_div(A.M, 64);
    const int nt = mt * ceil_div(A.N, 64) >= 128 ? 4 : mt * ceil_div(A.N, 32) >= 128 ? 2 : 1;
    if (A.M <= 32) return nt == 4 ? rows(Int<4>{}, Int<2>{}, Int<1>{}) : nt == 2 ? rows(Int<2>{}, Int<2>{}, Int<2>{}) : rows(Int<1>{}, Int<2>{}, Int<2>{});
    return nt == 4 ? rows(Int<4>{}, Int<4>{}, Int<1>{}) : nt == 2 ? rows(Int<2>{}, Int<4>{}, Int<1>{}) : rows(Int<1>{}, Int<4>{}, Int<1>{});
}

// Host-side checks of an observer call; the workgroup count on success.
lpq_status observe_args(const uint16_t* x, int64_t M, int64_t N, int observer, const float* state, const float* amax,
                        lpq_tensor* one, int64_t* units) {
    if (!state || !amax) return LPQ_ERR_NULL;
    if (!aligned(state, 4) || !aligned(amax, 4)) return LPQ_ERR_ALIGN;
    if (observer < LPQ_OBSERVER_MEMORYLESS_MINMAX || observer > LPQ_OBSERVER_MINMAX) return LPQ_ERR_ARG;
    *one = make_one(x, nullptr, nullptr, M, N);
    lpq_status st = check_tensor(NV_AMAX, *one, 0);   // same shape and alignment rules as the amax pass
    if (st != LPQ_OK) return st;
    *units = (M * N + chunk_elems<LPQ_AMAX_U>() - 1) / chunk_elems<LPQ_AMAX_U>();
    return *units > max_groups(kThreads) ? LPQ_ERR_SHAPE : LPQ_OK;
}

}  // namespace

// ---------------------------------------------------------------------------
// The allocation-free observer call keeps the control words of a call (batch
// keys and arrival counter) in a block the library holds, instead of in the
// caller's state.  Every device the library runs on holds its own copy of the
// block until the process ends.  All such calls on one device share it: each
// call re-arms it first, and calls that overlap on one device race.

static __device__ __align__(256) uint32_t scratch[kObsCtlWords];

namespace {

constexpr int kMaxScratchDevices = 64;
std::atomic<uint32_t*> g_scratch_ptr[kMaxScratchDevices];

inline lpq_status hip_failed(hipError_t e) {
    g_last_hip_error = (int)e;
    return LPQ_ERR_HIP;
}

// The device address of `scratch` on the device that `stream` runs on (the
// current device for the null stream).  It is looked up once per device, with
// that device current, and kept: on the host the name `scratch` is a stand-in,
// not a device address, and each device holds the block at its own address.
lpq_status scratch_on(hipStream_t stream, uint32_t** out) {
    int dev = 0;
    hipError_t e = stream ? hipStreamGetDevice(stream, &dev) : hipGetDevice(&dev);
    if (e != hipSuccess) return hip_failed(e);
    if (dev < 0 || dev >= kMaxScratchDevices) return hip_failed(hipErrorInvalidDevice);
    uint32_t* p = g_scratch_ptr[dev].load(std::memory_order_acquire);
    if (!p) {
        int cur = 0;
        if ((e = hipGetDevice(&cur)) != hipSuccess) return hip_failed(e);
        if (cur != dev && (e = hipSetDevice(dev)) != hipSuccess) return hip_failed(e);
        void* q = nullptr;
        e = hipGetSymbolAddress(&q, HIP_SYMBOL(scratch));
        if (cur != dev) {
            const hipError_t r = hipSetDevice(cur);
            if (e == hipSuccess) e = r;
        }
        if (e != hipSuccess) return hip_failed(e);
        if (!q) return hip_failed(hipErrorInvalidSymbol);
        p = static_cast<uint32_t*>(q);
        g_scratch_ptr[dev].store(p, std::memory_order_release);
    }
    *out = p;
    return LPQ_OK;
}

}  // namespace

extern "C" {

const char* lpq_status_string(lpq_status status) {
    switch (status) {
    case LPQ_OK: return "ok";
    case LPQ_ERR_NULL: return "a required pointer is NULL";
    case LPQ_ERR_SHAPE: return "invalid shape (M or N <= 0, N not a multiple of the block, or count <= 0)";
    case LPQ_ERR_ALIGN: return "a pointer is not aligned as required";
    case LPQ_ERR_GROUP: return "sibling-group index out of range";
    case LPQ_ERR_HIP: return "HIP launch failed (see lpq_last_hip_error)";
    case LPQ_ERR_ARG: return "invalid argument";
    default: return "unknown status";
    }
}

int lpq_last_hip_error(void) { return g_last_hip_error; }

int lpq_version(void) { return 10000; }

lpq_status lpq_quantize_fp8blk(const uint16_t* w, int64_t M, int64_t N, uint8_t* q, float* s, void* stream) {
    const lpq_tensor one = make_one(w, q, s, M, N);
    return single(fp8blk_quant_kind(&one, 1), one, nullptr, nullptr, stream);
}

lpq_status lpq_dequantize_fp8blk(const uint8_t* q, const float* s, int64_t M, int64_t N, uint16_t* y, void* stream) {
    const lpq_tensor one = make_one(q, y, const_cast<float*>(s), M, N);
    const bool flat = check_tensor(FP8BLK_DQF, one, 0) == LPQ_OK;   // with what FP8BLK_DQ asks for
    return single(flat ? FP8BLK_DQF : FP8BLK_DQ, one, nullptr, nullptr, stream);
}

lpq_status lpq_quantize_mxfp8(const uint16_t* w, int64_t M, int64_t N, uint8_t* q, uint8_t* e, void* stream) {
    return single(MXFP8_Q, make_one(w, q, e, M, N), nullptr, nullptr, stream);
}

lpq_status lpq_quantize_mxfp8_floor(const uint16_t* w, int64_t M, int64_t N, uint8_t* q, uint8_t* e, void* stream) {
    return single(MXFP8_QF, make_one(w, q, e, M, N), nullptr, nullptr, stream);
}

lpq_status lpq_quantize_mxfp8_floor_grouped(const lpq_tensor* host, const lpq_tensor* dev, int32_t n, void* stream) {
    return grouped(MXFP8_QF, host, dev, n, 0, nullptr, nullptr, stream);
}

lpq_status lpq_quantize_mxfp4(const uint16_t* w, int64_t M, int64_t N, uint8_t* p, uint8_t* e, void* stream) {
    return single(MXFP4_Q, make_one(w, p, e, M, N), nullptr, nullptr, stream);
}

lpq_status lpq_quantize_mxfp4_floor(const uint16_t* w, int64_t M, int64_t N, uint8_t* p, uint8_t* e, void* stream) {
    return single(MXFP4_QF, make_one(w, p, e, M, N), nullptr, nullptr, stream);
}

lpq_status lpq_dequantize_mxfp4(const uint8_t* p, const uint8_t* e, int64_t M, int64_t N, uint16_t* y, void* stream) {
    return single(MXFP4_DQ, make_one(p, y, const_cast<uint8_t*>(e), M, N), nullptr, nullptr, stream);
}

lpq_status lpq_mxfp4_qdq(const uint16_t* x, int64_t M, int64_t N, uint16_t* y, void* stream) {
    return single(MXFP4_QDQ, make_one(x, y, nullptr, M, N), nullptr, nullptr, stream);
}

lpq_status lpq_mxfp4_qdq_floor(const uint16_t* x, int64_t M, int64_t N, uint16_t* y, void* stream) {
    return single(MXFP4_QDQF, make_one(x, y, nullptr, M, N), nullptr, nullptr, stream);
}

lpq_status lpq_quantize_mxfp4_grouped(const lpq_tensor* host, const lpq_tensor* dev, int32_t n, void* stream) {
    return grouped(MXFP4_Q, host, dev, n, 0, nullptr, nullptr, stream);
}

lpq_status lpq_quantize_mxfp4_floor_grouped(const lpq_tensor* host, const lpq_tensor* dev, int32_t n, void* stream) {
    return grouped(MXFP4_QF, host, dev, n, 0, nullptr, nullptr, stream);
}

lpq_status lpq_dequantize_mxfp4_grouped(const lpq_tensor* host, const lpq_tensor* dev, int32_t n, void* stream) {
    return grouped(MXFP4_DQ, host, dev, n, 0, nullptr, nullptr, stream);
}

lpq_status lpq_mxfp4_qdq_grouped(const lpq_tensor* host, const lpq_tensor* dev, int32_t n, void* stream) {
    return grouped(MXFP4_QDQ, host, dev, n, 0, nullptr, nullptr, stream);
}

lpq_status lpq_mxfp4_qdq_floor_grouped(const lpq_tensor* host, const lpq_tensor* dev, int32_t n, void* stream) {
    return grouped(MXFP4_QDQF, host, dev, n, 0, nullptr, nullptr, stream);
}

lpq_status lpq_quantize_mxfp8_transposed(const uint16_t* w, int64_t M, int64_t N, int floor_rule, uint8_t* q, uint8_t* e,
                                         uint8_t* qt, uint8_t* et, void* stream) {
    return mx_transpose<false>(w, M, N, floor_rule, q, e, qt, et, stream);
}

lpq_status lpq_quantize_mxfp4_transposed(const uint16_t* w, int64_t M, int64_t N, int floor_rule, uint8_t* p, uint8_t* e,
                                         uint8_t* pt, uint8_t* et, void* stream) {
    return mx_transpose<true>(w, M, N, floor_rule, p, e, pt, et, stream);
}

lpq_status lpq_rmsnorm(const uint16_t* x, const uint16_t* residual, const uint16_t* gamma, float eps, int64_t M, int64_t N,
                       uint16_t* h, float* rstd, uint16_t* y, void* stream) {
    if (N <= 0 || N > kNormMaxN) return LPQ_ERR_SHAPE;
    return rmsnorm(NormArgs{x, residual, gamma, h, y, rstd, nullptr, nullptr, M, (int32_t)N, eps}, stream);
}

lpq_status lpq_rmsnorm_mxfp8(const uint16_t* x, const uint16_t* residual, const uint16_t* gamma, float eps, int64_t M, int64_t N,
                             uint16_t* h, float* rstd, uint16_t* y, uint8_t* q, uint8_t* e, void* stream) {
    if (N <= 0 || N > kNormMaxN) return LPQ_ERR_SHAPE;
    if (!q || !e) return LPQ_ERR_NULL;
    return rmsnorm(NormArgs{x, residual, gamma, h, y, rstd, q, e, M, (int32_t)N, eps}, stream);
}

int64_t lpq_rmsnorm_backward_workspace(int64_t M, int64_t N) {
    return norm_shape(M, N) == LPQ_OK ? 4 * norm_grad_groups(M, N) * N : 0;
}

lpq_status lpq_rmsnorm_backward(const uint16_t* dy, const uint16_t* h, const uint16_t* gamma, const float* rstd,
                                const uint16_t* dres, int64_t M, int64_t N, uint16_t* dx, float* dgamma, int accumulate,
                                void* workspace, int64_t workspace_bytes, void* stream) {
    if (N <= 0 || N > kNormMaxN) return LPQ_ERR_SHAPE;
    return rmsnorm_grad(NormGradArgs{dy, h, gamma, dres, rstd, dx, nullptr, M, (int32_t)N}, dgamma, accumulate, workspace,
                        workspace_bytes, stream);
}

lpq_status lpq_mx_matmul(const uint8_t* a, const uint8_t* ae, int a_format, const uint8_t* b, const uint8_t* be, int b_format,
                         int64_t M, int64_t N, int64_t K, void* y, int y_type, void* stream) {
    const int64_t most = int64_t(1) << 30;   // indexes along a row, some steps past its end too, stay 32-bit
    if (M <= 0 || N <= 0 || K <= 0 || K % 32 || M > most || N > most || K > most) return LPQ_ERR_SHAPE;
    if (M > (int64_t(1) << 40) / N || M > (int64_t(1) << 40) / K || N > (int64_t(1) << 40) / K) return LPQ_ERR_SHAPE;
    if (!a || !ae || !b || !be || !y) return LPQ_ERR_NULL;
    const bool a4 = a_format == LPQ_MXFP4, b4 = b_format == LPQ_MXFP4;
    if ((!a4 && a_format != LPQ_MXFP8) || (!b4 && b_format != LPQ_MXFP8)) return LPQ_ERR_ARG;
    if (y_type != LPQ_BF16 && !(y_type == LPQ_F32 && a4 && b4)) return LPQ_ERR_ARG;
    if (!aligned(a, 16) || !aligned(b, 16) || !aligned(y, 16)) return LPQ_ERR_ALIGN;
    const int64_t ny = M * N * (y_type == LPQ_F32 ? 4 : 2);
    if (overlap(y, ny, a, M * K / (a4 ? 2 : 1)) || overlap(y, ny, ae, M * K / 32) || overlap(y, ny, b, N * K / (b4 ? 2 : 1)) ||
        overlap(y, ny, be, N * K / 32))
        return LPQ_ERR_ARG;
    const MatmulArgs A{a, ae, b, be, y, (int32_t)M, (int32_t)N, (int32_t)K, y_type == LPQ_F32};
    const hipStream_t s = (hipStream_t)stream;
    if (a4) return b4 ? mx_matmul<true, true>(A, s) : mx_matmul<true, false>(A, s);
    return b4 ? mx_matmul<false, true>(A, s) : mx_matmul<false, false>(A, s);
}

lpq_status lpq_nvfp4_global_scale_reciprocal(const float* group_amax, int32_t n_groups, float* out, void* stream) {
    if (!group_amax || !out) return LPQ_ERR_NULL;
    if (n_groups <= 0) return LPQ_ERR_SHAPE;
    if (!aligned(group_amax, 4) || !aligned(out, 4)) return LPQ_ERR_ALIGN;
    hipLaunchKernelGGL(k_global_scale_reciprocal, dim3((unsigned)((n_groups + kThreads - 1) / kThreads)), dim3(kThreads),
                       0, (hipStream_t)stream, group_amax, n_groups, out);
    return launched();
}

lpq_status lpq_nvfp4_global_scale(const float* amax, int32_t n, float* out, void* stream) {
    if (!amax || !out) return LPQ_ERR_NULL;
    if (n <= 0) return LPQ_ERR_SHAPE;
    if (!aligned(amax, 4) || !aligned(out, 4)) return LPQ_ERR_ALIGN;
    return global_scale(amax, n, out, 2688.0f, stream);
}

lpq_status lpq_observer_reset(float* state, void* stream) {
    if (!state) return LPQ_ERR_NULL;
    if (!aligned(state, 4)) return LPQ_ERR_ALIGN;
    hipLaunchKernelGGL(k_observer_reset, dim3(1), dim3(64), 0, (hipStream_t)stream, reinterpret_cast<uint32_t*>(state));
    return launched();
}

lpq_status lpq_nvfp4_observe(const uint16_t* x, int64_t M, int64_t N, int observer, float averaging_constant,
                             float* state, float* amax, void* stream) {
    lpq_tensor one;
    int64_t units = 0;
    const lpq_status st = observe_args(x, M, N, observer, state, amax, &one, &units);
    if (st != LPQ_OK) return st;
    hipLaunchKernelGGL((k_minmax<LPQ_AMAX_U>), dim3((unsigned)units), dim3(kThreads), 0, (hipStream_t)stream, one,
                       observer, averaging_constant, state, reinterpret_cast<uint32_t*>(state), amax);
    return launched();
}

lpq_status lpq_nvfp4_observe_noalloc(const uint16_t* x, int64_t M, int64_t N, int observer,
                                     float averaging_constant, float* state, float* amax, void* stream) {
    lpq_tensor one;
    int64_t units = 0;
    lpq_status st = observe_args(x, M, N, observer, state, amax, &one, &units);
    if (st != LPQ_OK) return st;
    uint32_t* ctl = nullptr;
    if ((st = scratch_on((hipStream_t)stream, &ctl)) != LPQ_OK) return st;
    hipLaunchKernelGGL(k_observer_arm, dim3(1), dim3(64), 0, (hipStream_t)stream, ctl);
    if ((st = launched()) != LPQ_OK) return st;
    hipLaunchKernelGGL((k_minmax<LPQ_AMAX_U>), dim3((unsigned)units), dim3(kThreads), 0, (hipStream_t)stream, one,
                       observer, averaging_constant, state, ctl, amax);
    return launched();
}

lpq_status lpq_dequantize_mxfp8(const uint8_t* q, const uint8_t* e, int64_t M, int64_t N, uint16_t* y, void* stream) {
    return single(MXFP8_DQ, make_one(q, y, const_cast<uint8_t*>(e), M, N), nullptr, nullptr, stream);
}

lpq_status lpq_nvfp4_amax(const uint16_t* w, int64_t M, int64_t N, float* amax, int accumulate, void* stream) {
    if (!amax) return LPQ_ERR_NULL;
    if (!aligned(amax, 4)) return LPQ_ERR_ALIGN;
    const lpq_tensor one = make_one(w, nullptr, nullptr, M, N);
    lpq_status st = check_tensor(NV_AMAX, one, 0);
    if (st != LPQ_OK) return st;
    if (!accumulate && (st = fill(amax, 1, 0.0f, stream)) != LPQ_OK) return st;
    return launch<lpq_tensor>(NV_AMAX, nullptr, nullptr, 0, one, nullptr, amax, (hipStream_t)stream);
}

lpq_status lpq_quantize_nvfp4(const uint16_t* w, int64_t M, int64_t N, const float* amax, uint8_t* p, uint8_t* s,
                              float* g, void* stream) {
    return nvfp4_single(NV_Q, w, M, N, amax, 448, p, s, g, stream);
}

lpq_status lpq_dequantize_nvfp4(const uint8_t* p, const uint8_t* s, const float* g, int64_t M, int64_t N, uint16_t* y,
                                void* stream) {
    if (!g) return LPQ_ERR_NULL;
    if (!aligned(g, 4)) return LPQ_ERR_ALIGN;
    return single(NV_DQ, make_one(p, y, const_cast<uint8_t*>(s), M, N), g, nullptr, stream);
}

lpq_status lpq_nvfp4_qdq(const uint16_t* x, int64_t M, int64_t N, const float* amax, uint16_t* y, void* stream) {
    return nvfp4_single(NV_QDQ, x, M, N, amax, 448, y, nullptr, nullptr, stream);
}

lpq_status lpq_quantize_nvfp4_ex(const uint16_t* w, int64_t M, int64_t N, const float* amax, int e4m3_max, uint8_t* p,
                                 uint8_t* s, float* g, void* stream) {
    return nvfp4_single(NV_Q, w, M, N, amax, e4m3_max, p, s, g, stream);
}

lpq_status lpq_nvfp4_qdq_ex(const uint16_t* x, int64_t M, int64_t N, const float* amax, int e4m3_max, uint16_t* y,
                            void* stream) {
    return nvfp4_single(NV_QDQ, x, M, N, amax, e4m3_max, y, nullptr, nullptr, stream);
}

lpq_status lpq_quantize_nvfp4_grouped_ex(const lpq_tensor* host, const lpq_tensor* dev, int32_t n, float* group_amax,
                                         int32_t n_groups, int amax_valid, int e4m3_max, float* group_g,
                                         void* stream) {
    return nvfp4_grouped(NV_Q, host, dev, n, group_amax, n_groups, amax_valid, e4m3_max, group_g, stream);
}

lpq_status lpq_nvfp4_qdq_grouped_ex(const lpq_tensor* host, const lpq_tensor* dev, int32_t n, float* group_amax,
                                    int32_t n_groups, int amax_valid, int e4m3_max, void* stream) {
    return nvfp4_grouped(NV_QDQ, host, dev, n, group_amax, n_groups, amax_valid, e4m3_max, nullptr, stream);
}

lpq_status lpq_quantize_fp8blk_grouped(const lpq_tensor* host, const lpq_tensor* dev, int32_t n, void* stream) {
    return grouped(fp8blk_quant_kind(host, n), host, dev, n, 0, nullptr, nullptr, stream);
}

lpq_status lpq_dequantize_fp8blk_grouped(const lpq_tensor* host, const lpq_tensor* dev, int32_t n, void* stream) {
    // the flat kernel when every tensor allows it, else the tile kernel for all
    bool flat = host != nullptr && n > 0;
    for (int32_t i = 0; flat && i < n; i++) flat = check_tensor(FP8BLK_DQF, host[i], 0) == LPQ_OK;
    return grouped(flat ? FP8BLK_DQF : FP8BLK_DQ, host, dev, n, 0, nullptr, nullptr, stream);
}

lpq_status lpq_quantize_mxfp8_grouped(const lpq_tensor* host, const lpq_tensor* dev, int32_t n, void* stream) {
    return grouped(MXFP8_Q, host, dev, n, 0, nullptr, nullptr, stream);
}

lpq_status lpq_dequantize_mxfp8_grouped(const lpq_tensor* host, const lpq_tensor* dev, int32_t n, void* stream) {
    return grouped(MXFP8_DQ, host, dev, n, 0, nullptr, nullptr, stream);
}

lpq_status lpq_nvfp4_amax_grouped(const lpq_tensor* host, const lpq_tensor* dev, int32_t n, float* group_amax,
                                  int32_t n_groups, int accumulate, void* stream) {
    if (!group_amax) return LPQ_ERR_NULL;
    if (n_groups <= 0) return LPQ_ERR_SHAPE;
    if (!aligned(group_amax, 4)) return LPQ_ERR_ALIGN;
    if (!host || !dev) return LPQ_ERR_NULL;
    if (n <= 0) return LPQ_ERR_SHAPE;
    for (int32_t i = 0; i < n; i++) {
        lpq_status st = check_tensor(NV_AMAX, host[i], n_groups);
        if (st != LPQ_OK) return st;
    }
    if (!accumulate) {
        lpq_status st = fill(group_amax, n_groups, 0.0f, stream);
        if (st != LPQ_OK) return st;
    }
    return grouped(NV_AMAX, host, dev, n, n_groups, nullptr, group_amax, stream);
}

lpq_status lpq_quantize_nvfp4_grouped(const lpq_tensor* host, const lpq_tensor* dev, int32_t n, float* group_amax,
                                      int32_t n_groups, int amax_valid, float* group_g, void* stream) {
    return nvfp4_grouped(NV_Q, host, dev, n, group_amax, n_groups, amax_valid, 448, group_g, stream);
}

lpq_status lpq_dequantize_nvfp4_grouped(const lpq_tensor* host, const lpq_tensor* dev, int32_t n,
                                        const float* group_g, int32_t n_groups, void* stream) {
    if (!group_g) return LPQ_ERR_NULL;
    if (n_groups <= 0) return LPQ_ERR_SHAPE;
    if (!aligned(group_g, 4)) return LPQ_ERR_ALIGN;
    return grouped(NV_DQ, host, dev, n, n_groups, group_g, nullptr, stream);
}

lpq_status lpq_nvfp4_qdq_grouped(const lpq_tensor* host, const lpq_tensor* dev, int32_t n, float* group_amax,
                                 int32_t n_groups, int amax_valid, void* stream) {
    return nvfp4_grouped(NV_QDQ, host, dev, n, group_amax, n_groups, amax_valid, 448, nullptr, stream);
}

lpq_status lpq_requantize_fp8blk(const uint8_t* q, const float* s, int64_t M, int64_t N, uint8_t* q_out, float* s_out,
                                 void* stream) {
    return single(RQ_FP8, make_requant(q, s, q_out, s_out, M, N), nullptr, nullptr, stream);
}

lpq_status lpq_requantize_fp8blk_grouped(const lpq_requant_tensor* host, const lpq_requant_tensor* dev, int32_t n,
                                         void* stream) {
    return grouped(RQ_FP8, host, dev, n, 0, nullptr, nullptr, stream);
}

lpq_status lpq_requantize_fp8blk_mxfp8(const uint8_t* q, const float* s, int64_t M, int64_t N, uint8_t* q_out,
                                       uint8_t* e_out, void* stream) {
    return single(RQ_MX, make_requant(q, s, q_out, e_out, M, N), nullptr, nullptr, stream);
}

lpq_status lpq_fp8blk_amax(const uint8_t* q, const float* s, int64_t M, int64_t N, float* amax, int accumulate,
                           void* stream) {
    if (!amax) return LPQ_ERR_NULL;
    if (!aligned(amax, 4)) return LPQ_ERR_ALIGN;
    const lpq_requant_tensor one = make_requant(q, s, nullptr, nullptr, M, N);
    lpq_status st = check_tensor(RQ_AMAX, one, 0);
    if (st != LPQ_OK) return st;
    if (!accumulate && (st = fill(amax, 1, 0.0f, stream)) != LPQ_OK) return st;
    return launch<lpq_requant_tensor>(RQ_AMAX, nullptr, nullptr, 0, one, nullptr, amax, (hipStream_t)stream);
}

lpq_status lpq_requantize_fp8blk_nvfp4(const uint8_t* q, const float* s, int64_t M, int64_t N, const float* amax,
                                       uint8_t* p, uint8_t* sb, float* g, void* stream) {
    if (!amax || !g) return LPQ_ERR_NULL;
    if (!aligned(amax, 4) || !aligned(g, 4)) return LPQ_ERR_ALIGN;
    return single(RQ_NV, make_requant(q, s, p, sb, M, N), amax, g, stream);
}

lpq_status lpq_requantize_fp8blk_mxfp8_grouped(const lpq_requant_tensor* host, const lpq_requant_tensor* dev,
                                               int32_t n, void* stream) {
    return grouped(RQ_MX, host, dev, n, 0, nullptr, nullptr, stream);
}

lpq_status lpq_fp8blk_amax_grouped(const lpq_requant_tensor* host, const lpq_requant_tensor* dev, int32_t n,
                                   float* group_amax, int32_t n_groups, int accumulate, void* stream) {
    if (!group_amax) return LPQ_ERR_NULL;
    if (n_groups <= 0) return LPQ_ERR_SHAPE;
    if (!aligned(group_amax, 4)) return LPQ_ERR_ALIGN;
    if (!host || !dev) return LPQ_ERR_NULL;
    if (n <= 0) return LPQ_ERR_SHAPE;
    for (int32_t i = 0; i < n; i++) {
        lpq_status st = check_tensor(RQ_AMAX, host[i], n_groups);
        if (st != LPQ_OK) return st;
    }
    if (!accumulate) {
        lpq_status st = fill(group_amax, n_groups, 0.0f, stream);
        if (st != LPQ_OK) return st;
    }
    return grouped(RQ_AMAX, host, dev, n, n_groups, nullptr, group_amax, stream);
}

lpq_status lpq_requantize_fp8blk_nvfp4_grouped(const lpq_requant_tensor* host, const lpq_requant_tensor* dev,
                                               int32_t n, const float* group_amax, int32_t n_groups,
                                               float* group_g, void* stream) {
    if (!group_amax || !group_g) return LPQ_ERR_NULL;
    if (n_groups <= 0) return LPQ_ERR_SHAPE;
    if (!aligned(group_amax, 4) || !aligned(group_g, 4)) return LPQ_ERR_ALIGN;
    return grouped(RQ_NV, host, dev, n, n_groups, group_amax, group_g, stream);
}

lpq_status lpq_quantize_int4(const uint16_t* w, int64_t M, int64_t N, int32_t group, uint8_t* p, float* s,
                             void* stream) {
    const int k = int4_kind(I4_Q32, I4_Q128, group);
    if (k < 0) return LPQ_ERR_ARG;
    return single((Kind)k, make_one(w, p, s, M, N), nullptr, nullptr, stream);
}

lpq_status lpq_dequantize_int4(const uint8_t* p, const float* s, int64_t M, int64_t N, int32_t group, uint16_t* y,
                               void* stream) {
    const int k = int4_kind(I4_DQ32, I4_DQ128, group);
    if (k < 0) return LPQ_ERR_ARG;
    return single((Kind)k, make_one(p, y, const_cast<float*>(s), M, N), nullptr, nullptr, stream);
}

lpq_status lpq_int4_qdq(const uint16_t* x, int64_t M, int64_t N, int32_t group, uint16_t* y, void* stream) {
    const int k = int4_kind(I4_QDQ32, I4_QDQ128, group);
    if (k < 0) return LPQ_ERR_ARG;
    return single((Kind)k, make_one(x, y, nullptr, M, N), nullptr, nullptr, stream);
}

lpq_status lpq_quantize_int4_grouped(const lpq_tensor* host, const lpq_tensor* dev, int32_t n, int32_t group,
                                     void* stream) {
    const int k = int4_kind(I4_Q32, I4_Q128, group);
    if (k < 0) return LPQ_ERR_ARG;
    return grouped((Kind)k, host, dev, n, 0, nullptr, nullptr, stream);
}

lpq_status lpq_dequantize_int4_grouped(const lpq_tensor* host, const lpq_tensor* dev, int32_t n, int32_t group,
                                       void* stream) {
    const int k = int4_kind(I4_DQ32, I4_DQ128, group);
    if (k < 0) return LPQ_ERR_ARG;
    return grouped((Kind)k, host, dev, n, 0, nullptr, nullptr, stream);
}

lpq_status lpq_int4_qdq_grouped(const lpq_tensor* host, const lpq_tensor* dev, int32_t n, int32_t group,
                                void* stream) {
    const int k = int4_kind(I4_QDQ32, I4_QDQ128, group);
    if (k < 0) return LPQ_ERR_ARG;
    return grouped((Kind)k, host, dev, n, 0, nullptr, nullptr, stream);
}

}  // extern "C"
