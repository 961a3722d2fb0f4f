// C ABI of libep_mi355x: argument checks on the host, then the gfx950 kernel launches.
// Every entry point is declared and documented in include/ep.h.
#include <stdint.h>
#include <stdio.h>

#include <mutex>
#include <string>

#include "ep.h"
#include "ep_expert.h"
#include "ep_internal.h"
#include "ep_product.h"

#ifndef EP_VERSION_STRING
#define EP_VERSION_STRING "0.1.0"
#endif

namespace ep {

LaunchLog &launch_log()
{
    thread_local LaunchLog log;
    return log;
}

}  // namespace ep

namespace {

thread_local std::string g_last_error;

int fail(int code, const std::string &what)
{
    g_last_error = what;
    return code;
}

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Shape rules common to every call. On failure returns a negative code and records why.
// Every entry point that launches kernels starts here, so this also clears the launch log.
int check_shape(const ep_shape_t *s, const char *fn)
{
    ep::launch_log().n = 0;
    std::string f(fn);
    if (!s) return fail(EP_ERR_INVALID, f + ": shape is NULL");
    if (s->T < 0 || s->H < 1 || s->E < 1 || s->K < 1 || s->C < 1 || s->R < 1)
        return fail(EP_ERR_INVALID, f + ": need T >= 0 and H, E, K, C, R >= 1");
    if (s->E % s->R != 0) return fail(EP_ERR_INVALID, f + ": E must be a multiple of R");
    if ((int64_t)s->T * s->K > INT32_MAX) return fail(EP_ERR_INVALID, f + ": T*K exceeds INT32_MAX");
    if ((int64_t)s->E * s->C > INT32_MAX) return fail(EP_ERR_INVALID, f + ": E*C exceeds INT32_MAX");
    return EP_OK;
}

// Limits of the dispatch and combine kernels: 16-byte rows, and the K pairs of a token staged
// in one workgroup's LDS.
int check_rows(const ep_shape_t *s, const char *fn, int h_multiple)
{
    if (s->H % h_multiple != 0)
        return fail(EP_ERR_UNSUPPORTED, std::string(fn) + ": H must be a multiple of " +
                                            std::to_string(h_multiple));
    if (s->K > EP_MAX_TOPK)
        return fail(EP_ERR_UNSUPPORTED, std::string(fn) + ": K exceeds EP_MAX_TOPK");
    return EP_OK;
}

int hip_status(hipError_t e, const char *fn)
{
    if (e == hipSuccess) {
        g_last_error.clear();
        return EP_OK;
    }
    return fail(EP_ERR_HIP, std::string(fn) + ": " + hipGetErrorName(e) + ": " + hipGetErrorString(e));
}

// Checks shared by every call that computes the layout.
int check_layout_args(const ep_shape_t *shape, const int32_t *topk_idx, const int32_t *slot,
                      const int32_t *expert_count, const int32_t *expert_offset,
                      const int32_t *stats, const char *fn)
{
    const std::string f(fn);
    if (int rc = check_shape(shape, fn)) return rc;
    if (shape->E > EP_MAX_EXPERTS) return fail(EP_ERR_UNSUPPORTED, f + ": E exceeds EP_MAX_EXPERTS");
    const bool empty = (int64_t)shape->T * shape->K == 0;
    if ((!empty && (!topk_idx || !slot)) || !expert_count || !expert_offset || !stats)
        return fail(EP_ERR_INVALID, f + ": NULL required pointer");
    if (!aligned(topk_idx, 16))
        return fail(EP_ERR_ALIGN, f + ": topk_idx must be 16-byte aligned");
    return EP_OK;
}

// Limits of the two-stage calls: ranks as 64-bit sets, staging rows r*T + p in int32, expert
// ids below EP_MAX_EXPERTS (the rank of an id is found by a multiply exact up to there).
int check_ranks(const ep_shape_t *s, const char *fn)
{
    if (s->R > EP_MAX_RANKS)
        return fail(EP_ERR_UNSUPPORTED, std::string(fn) + ": R exceeds EP_MAX_RANKS");
    if (s->E > EP_MAX_EXPERTS)
        return fail(EP_ERR_UNSUPPORTED, std::string(fn) + ": E exceeds EP_MAX_EXPERTS");
    if ((int64_t)s->R * s->T > INT32_MAX)
        return fail(EP_ERR_UNSUPPORTED, std::string(fn) + ": R*T exceeds INT32_MAX");
    return EP_OK;
}

}  // namespace

extern "C" {

int ep_layout(const ep_shape_t *shape, const int32_t *topk_idx, int32_t *slot,
              int32_t *expert_count, int32_t *expert_offset, int32_t *rank_count,
              int32_t *rank_offset, int32_t *stats, hipStream_t stream)
{
    if (int rc = check_layout_args(shape, topk_idx, slot, expert_count, expert_offset, stats,
                                   "ep_layout"))
        return rc;
    const ep::LayoutOut o{slot, expert_count, expert_offset, rank_count, rank_offset, stats};
    return hip_status(ep::launch_layout(*shape, topk_idx, o, stream), "ep_layout");
}

int ep_layout_dispatch(const ep_shape_t *shape, const uint16_t *x, const int32_t *topk_idx,
                       int32_t *slot, int32_t *expert_count, int32_t *expert_offset,
                       int32_t *rank_count, int32_t *rank_offset, int32_t *stats,
                       uint16_t *recv, hipStream_t stream)
{
    if (int rc = check_layout_args(shape, topk_idx, slot, expert_count, expert_offset, stats,
                                   "ep_layout_dispatch"))
        return rc;
    if (int rc = check_rows(shape, "ep_layout_dispatch", 8)) return rc;
    if (shape->T > 0 && (!x || !recv))
        return fail(EP_ERR_INVALID, "ep_layout_dispatch: NULL required pointer");
    if (!aligned(x, 16) || !aligned(recv, 16))
        return fail(EP_ERR_ALIGN, "ep_layout_dispatch: x and recv must be 16-byte aligned");
    const ep::LayoutOut o{slot, expert_count, expert_offset, rank_count, rank_offset, stats};
    return hip_status(ep::launch_layout_dispatch_bf16(*shape, x, topk_idx, o, recv, stream),
                      "ep_layout_dispatch");
}

int ep_layout_dispatch_fp8(const ep_shape_t *shape, const uint16_t *x, const int32_t *topk_idx,
                           int32_t *slot, int32_t *expert_count, int32_t *expert_offset,
                           int32_t *rank_count, int32_t *rank_offset, int32_t *stats,
                           uint8_t *recv_q, float *recv_scale, hipStream_t stream)
{
    if (int rc = check_layout_args(shape, topk_idx, slot, expert_count, expert_offset, stats,
                                   "ep_layout_dispatch_fp8"))
        return rc;
    if (int rc = check_rows(shape, "ep_layout_dispatch_fp8", EP_FP8_BLOCK)) return rc;
    if (shape->T > 0 && (!x || !recv_q || !recv_scale))
        return fail(EP_ERR_INVALID, "ep_layout_dispatch_fp8: NULL required pointer");
    if (!aligned(x, 16) || !aligned(recv_q, 16) || !aligned(recv_scale, 4))
        return fail(EP_ERR_ALIGN, "ep_layout_dispatch_fp8: x and recv_q must be 16-byte aligned, "
                                  "recv_scale 4-byte aligned");
    const ep::LayoutOut o{slot, expert_count, expert_offset, rank_count, rank_offset, stats};
    return hip_status(ep::launch_layout_dispatch_fp8(*shape, x, topk_idx, o, recv_q, recv_scale,
                                                     stream),
                      "ep_layout_dispatch_fp8");
}

namespace {

// The static scratch of ep_layout_dispatch_noalloc: device memory of the library itself, one
// copy per GPU, held until the process ends. In host code `scratch` is only a stand-in for the
// symbol; its device address on the current GPU comes from hipGetSymbolAddress, once per
// device, and only that address is passed to kernels.
constexpr size_t kScratchBytes = size_t(1) << 20;
__device__ __align__(256) int32_t scratch[kScratchBytes / sizeof(int32_t)];

constexpr int kScratchDevices = 64;
void *g_scratch_ptr[kScratchDevices];
hipError_t g_scratch_status[kScratchDevices];
std::once_flag g_scratch_once[kScratchDevices];

// This device's address of `scratch` (looked up on the first call on the device, with the
// device current).
int scratch_on_current_device(void **ptr, const char *fn)
{
    int dev = -1;
    if (hipError_t e = hipGetDevice(&dev)) return hip_status(e, fn);
    if (dev < 0 || dev >= kScratchDevices)
        return fail(EP_ERR_UNSUPPORTED, std::string(fn) + ": device ordinal " +
                                            std::to_string(dev) + " beyond the library's " +
                                            std::to_string(kScratchDevices));
    std::call_once(g_scratch_once[dev], [dev] {
        g_scratch_status[dev] = hipGetSymbolAddress(&g_scratch_ptr[dev], HIP_SYMBOL(scratch));
    });
    if (g_scratch_status[dev] != hipSuccess) return hip_status(g_scratch_status[dev], fn);
    *ptr = g_scratch_ptr[dev];
    return EP_OK;
}

// The workspace of the chunked layout: present, large enough and 16-byte aligned.
int check_workspace(const ep_shape_t *shape, const void *workspace, size_t workspace_bytes,
                    const char *fn)
{
    const size_t need = ep::layout_workspace_bytes(*shape);
    if (need > 0 && !workspace) return fail(EP_ERR_INVALID, std::string(fn) + ": workspace is NULL");
    if (workspace_bytes < need)
        return fail(EP_ERR_INVALID, std::string(fn) + ": workspace_bytes " +
                                        std::to_string(workspace_bytes) + " below the " +
                                        std::to_string(need) + " this shape needs");
    if (!aligned(workspace, 16))
        return fail(EP_ERR_ALIGN, std::string(fn) + ": workspace must be 16-byte aligned");
    return EP_OK;
}

}  // namespace

size_t ep_layout_workspace_bytes(const ep_shape_t *shape)
{
    if (!shape || shape->T < 0 || shape->K < 1 || shape->E < 1 ||
        (int64_t)shape->T * shape->K > INT32_MAX)
        return 0;
    return ep::layout_workspace_bytes(*shape);
}

int ep_layout_dispatch_ws(const ep_shape_t *shape, const uint16_t *x, const int32_t *topk_idx,
                          int32_t *slot, int32_t *expert_count, int32_t *expert_offset,
                          int32_t *rank_count, int32_t *rank_offset, int32_t *stats,
                          uint16_t *recv, void *workspace, size_t workspace_bytes,
                          hipStream_t stream)
{
    const char *fn = "ep_layout_dispatch_ws";
    if (int rc = check_layout_args(shape, topk_idx, slot, expert_count, expert_offset, stats, fn))
        return rc;
    if (int rc = check_rows(shape, fn, 8)) return rc;
    if (shape->T > 0 && (!x || !recv))
        return fail(EP_ERR_INVALID, "ep_layout_dispatch_ws: NULL required pointer");
    if (!aligned(x, 16) || !aligned(recv, 16))
        return fail(EP_ERR_ALIGN, "ep_layout_dispatch_ws: x and recv must be 16-byte aligned");
    if (int rc = check_workspace(shape, workspace, workspace_bytes, fn)) return rc;
    const ep::LayoutOut o{slot, expert_count, expert_offset, rank_count, rank_offset, stats};
    return hip_status(ep::launch_layout_dispatch_bf16_chunked(
                          *shape, x, topk_idx, o, recv, static_cast<int32_t *>(workspace), stream),
                      fn);
}

int ep_layout_dispatch_fp8_ws(const ep_shape_t *shape, const uint16_t *x,
                              const int32_t *topk_idx, int32_t *slot, int32_t *expert_count,
                              int32_t *expert_offset, int32_t *rank_count, int32_t *rank_offset,
                              int32_t *stats, uint8_t *recv_q, float *recv_scale,
                              void *workspace, size_t workspace_bytes, hipStream_t stream)
{
    const char *fn = "ep_layout_dispatch_fp8_ws";
    if (int rc = check_layout_args(shape, topk_idx, slot, expert_count, expert_offset, stats, fn))
        return rc;
    if (int rc = check_rows(shape, fn, EP_FP8_BLOCK)) return rc;
    if (shape->T > 0 && (!x || !recv_q || !recv_scale))
        return fail(EP_ERR_INVALID, "ep_layout_dispatch_fp8_ws: NULL required pointer");
    if (!aligned(x, 16) || !aligned(recv_q, 16) || !aligned(recv_scale, 4))
        return fail(EP_ERR_ALIGN, "ep_layout_dispatch_fp8_ws: x and recv_q must be 16-byte "
                                  "aligned, recv_scale 4-byte aligned");
    if (int rc = check_workspace(shape, workspace, workspace_bytes, fn)) return rc;
    const ep::LayoutOut o{slot, expert_count, expert_offset, rank_count, rank_offset, stats};
    return hip_status(ep::launch_layout_dispatch_fp8_chunked(*shape, x, topk_idx, o, recv_q,
                                                             recv_scale,
                                                             static_cast<int32_t *>(workspace),
                                                             stream),
                      fn);
}

int ep_layout_dispatch_noalloc(const ep_shape_t *shape, const uint16_t *x,
                               const int32_t *topk_idx, int32_t *slot, int32_t *expert_count,
                               int32_t *expert_offset, int32_t *rank_count, int32_t *rank_offset,
                               int32_t *stats, uint16_t *recv, hipStream_t stream)
{
    const char *fn = "ep_layout_dispatch_noalloc";
    if (int rc = check_layout_args(shape, topk_idx, slot, expert_count, expert_offset, stats, fn))
        return rc;
    if (int rc = check_rows(shape, fn, 8)) return rc;
    if (shape->T > 0 && (!x || !recv))
        return fail(EP_ERR_INVALID, "ep_layout_dispatch_noalloc: NULL required pointer");
    if (!aligned(x, 16) || !aligned(recv, 16))
        return fail(EP_ERR_ALIGN, "ep_layout_dispatch_noalloc: x and recv must be 16-byte aligned");
    const size_t need = ep::layout_workspace_bytes(*shape);
    if (need > kScratchBytes)
        return fail(EP_ERR_UNSUPPORTED, "ep_layout_dispatch_noalloc: this shape needs " +
                                            std::to_string(need) +
                                            " bytes of workspace, more than the library's "
                                            "static scratch of " +
                                            std::to_string(kScratchBytes) +
                                            " (use ep_layout_dispatch_ws)");
    void *ws = nullptr;
    if (int rc = scratch_on_current_device(&ws, fn)) return rc;
    const ep::LayoutOut o{slot, expert_count, expert_offset, rank_count, rank_offset, stats};
    return hip_status(ep::launch_layout_dispatch_bf16_chunked(*shape, x, topk_idx, o, recv,
                                                              static_cast<int32_t *>(ws), stream),
                      fn);
}

int ep_dispatch(const ep_shape_t *shape, const uint16_t *x, const int32_t *topk_idx,
                const int32_t *slot, uint16_t *recv, hipStream_t stream)
{
    if (int rc = check_shape(shape, "ep_dispatch")) return rc;
    if (int rc = check_rows(shape, "ep_dispatch", 8)) return rc;
    if (shape->T == 0) return hip_status(hipSuccess, "ep_dispatch");
    if (!x || !topk_idx || !slot || !recv)
        return fail(EP_ERR_INVALID, "ep_dispatch: NULL required pointer");
    if (!aligned(x, 16) || !aligned(recv, 16))
        return fail(EP_ERR_ALIGN, "ep_dispatch: x and recv must be 16-byte aligned");
    return hip_status(ep::launch_dispatch_bf16(*shape, x, topk_idx, slot, recv, stream),
                      "ep_dispatch");
}

int ep_dispatch_fp8(const ep_shape_t *shape, const uint16_t *x, const int32_t *topk_idx,
                    const int32_t *slot, uint8_t *recv_q, float *recv_scale, hipStream_t stream)
{
    if (int rc = check_shape(shape, "ep_dispatch_fp8")) return rc;
    if (int rc = check_rows(shape, "ep_dispatch_fp8", EP_FP8_BLOCK)) return rc;
    if (shape->T == 0) return hip_status(hipSuccess, "ep_dispatch_fp8");
    if (!x || !topk_idx || !slot || !recv_q || !recv_scale)
        return fail(EP_ERR_INVALID, "ep_dispatch_fp8: NULL required pointer");
    if (!aligned(x, 16) || !aligned(recv_q, 16) || !aligned(recv_scale, 4))
        return fail(EP_ERR_ALIGN, "ep_dispatch_fp8: x and recv_q must be 16-byte aligned, "
                                  "recv_scale 4-byte aligned");
    return hip_status(ep::launch_dispatch_fp8(*shape, x, topk_idx, slot, recv_q, recv_scale,
                                              stream),
                      "ep_dispatch_fp8");
}

int ep_combine(const ep_shape_t *shape, const uint16_t *y, const int32_t *topk_idx,
               const int32_t *slot, const float *topk_w, uint16_t *out, hipStream_t stream)
{
    if (int rc = check_shape(shape, "ep_combine")) return rc;
    if (int rc = check_rows(shape, "ep_combine", 8)) return rc;
    if (shape->T == 0) return hip_status(hipSuccess, "ep_combine");
    if (!y || !topk_idx || !slot || !topk_w || !out)
        return fail(EP_ERR_INVALID, "ep_combine: NULL required pointer");
    if (!aligned(y, 16) || !aligned(out, 16))
        return fail(EP_ERR_ALIGN, "ep_combine: y and out must be 16-byte aligned");
    return hip_status(ep::launch_combine(*shape, y, topk_idx, slot, topk_w, out, stream),
                      "ep_combine");
}

int ep_rank_layout(const ep_shape_t *shape, const int32_t *topk_idx, int32_t *rank_slot,
                   int32_t *rank_tokens, hipStream_t stream)
{
    const char *fn = "ep_rank_layout";
    if (int rc = check_shape(shape, fn)) return rc;
    if (int rc = check_ranks(shape, fn)) return rc;
    if ((shape->T > 0 && (!topk_idx || !rank_slot)) || !rank_tokens)
        return fail(EP_ERR_INVALID, "ep_rank_layout: NULL required pointer");
    if (!aligned(topk_idx, 16) || !aligned(rank_slot, 16))
        return fail(EP_ERR_ALIGN, "ep_rank_layout: topk_idx and rank_slot must be 16-byte aligned");
    return hip_status(ep::launch_rank_layout(*shape, topk_idx, rank_slot, rank_tokens, stream),
                      fn);
}

int ep_dispatch_ranks(const ep_shape_t *shape, const uint16_t *x, const int32_t *rank_slot,
                      uint16_t *stage, hipStream_t stream)
{
    const char *fn = "ep_dispatch_ranks";
    if (int rc = check_shape(shape, fn)) return rc;
    if (int rc = check_rows(shape, fn, 8)) return rc;
    if (int rc = check_ranks(shape, fn)) return rc;
    if (shape->T == 0) return hip_status(hipSuccess, fn);
    if (!x || !rank_slot || !stage) return fail(EP_ERR_INVALID, "ep_dispatch_ranks: NULL required pointer");
    if (!aligned(x, 16) || !aligned(stage, 16))
        return fail(EP_ERR_ALIGN, "ep_dispatch_ranks: x and stage must be 16-byte aligned");
    return hip_status(ep::launch_dispatch_ranks_bf16(*shape, x, rank_slot, stage, stream), fn);
}

int ep_dispatch_ranks_fp8(const ep_shape_t *shape, const uint16_t *x, const int32_t *rank_slot,
                          uint8_t *stage_q, float *stage_scale, hipStream_t stream)
{
    const char *fn = "ep_dispatch_ranks_fp8";
    if (int rc = check_shape(shape, fn)) return rc;
    if (int rc = check_rows(shape, fn, EP_FP8_BLOCK)) return rc;
    if (int rc = check_ranks(shape, fn)) return rc;
    if (shape->T == 0) return hip_status(hipSuccess, fn);
    if (!x || !rank_slot || !stage_q || !stage_scale)
        return fail(EP_ERR_INVALID, "ep_dispatch_ranks_fp8: NULL required pointer");
    if (!aligned(x, 16) || !aligned(stage_q, 16) || !aligned(stage_scale, 4))
        return fail(EP_ERR_ALIGN, "ep_dispatch_ranks_fp8: x and stage_q must be 16-byte aligned, "
                                  "stage_scale 4-byte aligned");
    return hip_status(ep::launch_dispatch_ranks_fp8(*shape, x, rank_slot, stage_q, stage_scale,
                                                    stream),
                      fn);
}

int ep_rank_layout_dispatch(const ep_shape_t *shape, const uint16_t *x, const int32_t *topk_idx,
                            int32_t *rank_slot, int32_t *rank_tokens, uint16_t *stage,
                            hipStream_t stream)
{
    const char *fn = "ep_rank_layout_dispatch";
    if (int rc = check_shape(shape, fn)) return rc;
    if (int rc = check_rows(shape, fn, 8)) return rc;
    if (int rc = check_ranks(shape, fn)) return rc;
    if ((shape->T > 0 && (!x || !topk_idx || !rank_slot || !stage)) || !rank_tokens)
        return fail(EP_ERR_INVALID, "ep_rank_layout_dispatch: NULL required pointer");
    if (!aligned(topk_idx, 16) || !aligned(x, 16) || !aligned(stage, 16))
        return fail(EP_ERR_ALIGN, "ep_rank_layout_dispatch: topk_idx, x and stage must be "
                                  "16-byte aligned");
    return hip_status(ep::launch_rank_layout_dispatch_bf16(*shape, x, topk_idx, rank_slot,
                                                           rank_tokens, stage, stream),
                      fn);
}

int ep_rank_layout_dispatch_fp8(const ep_shape_t *shape, const uint16_t *x,
                                const int32_t *topk_idx, int32_t *rank_slot,
                                int32_t *rank_tokens, uint8_t *stage_q, float *stage_scale,
                                hipStream_t stream)
{
    const char *fn = "ep_rank_layout_dispatch_fp8";
    if (int rc = check_shape(shape, fn)) return rc;
    if (int rc = check_rows(shape, fn, EP_FP8_BLOCK)) return rc;
    if (int rc = check_ranks(shape, fn)) return rc;
    if ((shape->T > 0 && (!x || !topk_idx || !rank_slot || !stage_q || !stage_scale)) ||
        !rank_tokens)
        return fail(EP_ERR_INVALID, "ep_rank_layout_dispatch_fp8: NULL required pointer");
    if (!aligned(topk_idx, 16) || !aligned(x, 16) || !aligned(stage_q, 16) ||
        !aligned(stage_scale, 4))
        return fail(EP_ERR_ALIGN, "ep_rank_layout_dispatch_fp8: topk_idx, x and stage_q must be "
                                  "16-byte aligned, stage_scale 4-byte aligned");
    return hip_status(ep::launch_rank_layout_dispatch_fp8(*shape, x, topk_idx, rank_slot,
                                                          rank_tokens, stage_q, stage_scale,
                                                          stream),
                      fn);
}

int ep_dispatch_expand(const ep_shape_t *shape, const uint16_t *stage, const int32_t *topk_idx,
                       const int32_t *slot, const int32_t *rank_slot, uint16_t *recv,
                       hipStream_t stream)
{
    const char *fn = "ep_dispatch_expand";
    if (int rc = check_shape(shape, fn)) return rc;
    if (int rc = check_rows(shape, fn, 8)) return rc;
    if (int rc = check_ranks(shape, fn)) return rc;
    if (shape->T == 0) return hip_status(hipSuccess, fn);
    if (!stage || !topk_idx || !slot || !rank_slot || !recv)
        return fail(EP_ERR_INVALID, "ep_dispatch_expand: NULL required pointer");
    if (!aligned(stage, 16) || !aligned(recv, 16))
        return fail(EP_ERR_ALIGN, "ep_dispatch_expand: stage and recv must be 16-byte aligned");
    return hip_status(ep::launch_dispatch_expand_bf16(*shape, stage, topk_idx, slot, rank_slot,
                                                      recv, stream),
                      fn);
}

int ep_layout_dispatch_expand(const ep_shape_t *shape, const uint16_t *stage,
                              const int32_t *topk_idx, const int32_t *rank_slot, int32_t *slot,
                              int32_t *expert_count, int32_t *expert_offset, int32_t *rank_count,
                              int32_t *rank_offset, int32_t *stats, uint16_t *recv,
                              hipStream_t stream)
{
    const char *fn = "ep_layout_dispatch_expand";
    if (int rc = check_layout_args(shape, topk_idx, slot, expert_count, expert_offset, stats, fn))
        return rc;
    if (int rc = check_rows(shape, fn, 8)) return rc;
    if (int rc = check_ranks(shape, fn)) return rc;
    if (shape->T > 0 && (!stage || !rank_slot || !recv))
        return fail(EP_ERR_INVALID, "ep_layout_dispatch_expand: NULL required pointer");
    if (!aligned(stage, 16) || !aligned(recv, 16))
        return fail(EP_ERR_ALIGN,
                    "ep_layout_dispatch_expand: stage and recv must be 16-byte aligned");
    const ep::LayoutOut o{slot, expert_count, expert_offset, rank_count, rank_offset, stats};
    return hip_status(
        ep::launch_layout_expand_bf16(*shape, stage, topk_idx, rank_slot, o, recv, stream), fn);
}

int ep_layout_dispatch_expand_fp8(const ep_shape_t *shape, const uint8_t *stage_q,
                                  const float *stage_scale, const int32_t *topk_idx,
                                  const int32_t *rank_slot, int32_t *slot, int32_t *expert_count,
                                  int32_t *expert_offset, int32_t *rank_count,
                                  int32_t *rank_offset, int32_t *stats, uint8_t *recv_q,
                                  float *recv_scale, hipStream_t stream)
{
    const char *fn = "ep_layout_dispatch_expand_fp8";
    if (int rc = check_layout_args(shape, topk_idx, slot, expert_count, expert_offset, stats, fn))
        return rc;
    if (int rc = check_rows(shape, fn, EP_FP8_BLOCK)) return rc;
    if (int rc = check_ranks(shape, fn)) return rc;
    if (shape->T > 0 && (!stage_q || !stage_scale || !rank_slot || !recv_q || !recv_scale))
        return fail(EP_ERR_INVALID, "ep_layout_dispatch_expand_fp8: NULL required pointer");
    if (!aligned(stage_q, 16) || !aligned(recv_q, 16) || !aligned(stage_scale, 4) ||
        !aligned(recv_scale, 4))
        return fail(EP_ERR_ALIGN, "ep_layout_dispatch_expand_fp8: stage_q and recv_q must be "
                                  "16-byte aligned, the scales 4-byte aligned");
    const ep::LayoutOut o{slot, expert_count, expert_offset, rank_count, rank_offset, stats};
    return hip_status(ep::launch_layout_expand_fp8(*shape, stage_q, stage_scale, topk_idx,
                                                   rank_slot, o, recv_q, recv_scale, stream),
                      fn);
}

int ep_dispatch_expand_fp8(const ep_shape_t *shape, const uint8_t *stage_q,
                           const float *stage_scale, const int32_t *topk_idx,
                           const int32_t *slot, const int32_t *rank_slot, uint8_t *recv_q,
                           float *recv_scale, hipStream_t stream)
{
    const char *fn = "ep_dispatch_expand_fp8";
    if (int rc = check_shape(shape, fn)) return rc;
    if (int rc = check_rows(shape, fn, EP_FP8_BLOCK)) return rc;
    if (int rc = check_ranks(shape, fn)) return rc;
    if (shape->T == 0) return hip_status(hipSuccess, fn);
    if (!stage_q || !stage_scale || !topk_idx || !slot || !rank_slot || !recv_q || !recv_scale)
        return fail(EP_ERR_INVALID, "ep_dispatch_expand_fp8: NULL required pointer");
    if (!aligned(stage_q, 16) || !aligned(recv_q, 16) || !aligned(stage_scale, 4) ||
        !aligned(recv_scale, 4))
        return fail(EP_ERR_ALIGN, "ep_dispatch_expand_fp8: stage_q and recv_q must be 16-byte "
                                  "aligned, the scale buffers 4-byte aligned");
    return hip_status(ep::launch_dispatch_expand_fp8(*shape, stage_q, stage_scale, topk_idx, slot,
                                                     rank_slot, recv_q, recv_scale, stream),
                      fn);
}

int ep_combine_ranks(const ep_shape_t *shape, const uint16_t *y, const int32_t *topk_idx,
                     const int32_t *slot, const int32_t *rank_slot, const float *topk_w,
                     uint16_t *part, hipStream_t stream)
{
    const char *fn = "ep_combine_ranks";
    if (int rc = check_shape(shape, fn)) return rc;
    if (int rc = check_rows(shape, fn, 8)) return rc;
    if (int rc = check_ranks(shape, fn)) return rc;
    if (shape->T == 0) return hip_status(hipSuccess, fn);
    if (!y || !topk_idx || !slot || !rank_slot || !topk_w || !part)
        return fail(EP_ERR_INVALID, "ep_combine_ranks: NULL required pointer");
    if (!aligned(y, 16) || !aligned(part, 16))
        return fail(EP_ERR_ALIGN, "ep_combine_ranks: y and part must be 16-byte aligned");
    return hip_status(ep::launch_combine_ranks(*shape, y, topk_idx, slot, rank_slot, topk_w,
                                               part, stream),
                      fn);
}

int ep_combine_reduce(const ep_shape_t *shape, const uint16_t *part, const int32_t *rank_slot,
                      uint16_t *out, hipStream_t stream)
{
    const char *fn = "ep_combine_reduce";
    if (int rc = check_shape(shape, fn)) return rc;
    if (int rc = check_rows(shape, fn, 8)) return rc;
    if (int rc = check_ranks(shape, fn)) return rc;
    if (shape->T == 0) return hip_status(hipSuccess, fn);
    if (!part || !rank_slot || !out)
        return fail(EP_ERR_INVALID, "ep_combine_reduce: NULL required pointer");
    if (!aligned(part, 16) || !aligned(out, 16))
        return fail(EP_ERR_ALIGN, "ep_combine_reduce: part and out must be 16-byte aligned");
    return hip_status(ep::launch_combine_reduce(*shape, part, rank_slot, out, stream), fn);
}

int ep_layout_packed(const ep_shape_t *shape, int32_t alignment, const int32_t *topk_idx,
                     int32_t *slot, int32_t *expert_count, int32_t *packed_offset,
                     int32_t *rank_count, int32_t *rank_offset, int32_t *stats,
                     hipStream_t stream)
{
    const char *fn = "ep_layout_packed";
    if (int rc = check_layout_args(shape, topk_idx, slot, expert_count, packed_offset, stats, fn))
        return rc;
    if (alignment < 1) return fail(EP_ERR_INVALID, "ep_layout_packed: alignment must be >= 1");
    if ((int64_t)shape->E * ((int64_t)shape->C + alignment - 1) > INT32_MAX)
        return fail(EP_ERR_UNSUPPORTED, "ep_layout_packed: E*(C + alignment - 1) exceeds INT32_MAX");
    ep::LayoutOut o{slot, expert_count, packed_offset, rank_count, rank_offset, stats};
    o.offset_end = packed_offset + shape->E;
    o.align = alignment;
    return hip_status(ep::launch_layout(*shape, topk_idx, o, stream), fn);
}

namespace {

int check_packed(const ep_shape_t *shape, int32_t rows, const int32_t *packed_offset,
                 const char *fn, int h_multiple)
{
    if (int rc = check_shape(shape, fn)) return rc;
    if (int rc = check_rows(shape, fn, h_multiple)) return rc;
    if (rows < 0) return fail(EP_ERR_INVALID, std::string(fn) + ": rows must be >= 0");
    if (shape->T > 0 && !packed_offset)
        return fail(EP_ERR_INVALID, std::string(fn) + ": NULL required pointer");
    return EP_OK;
}

}  // namespace

namespace {

// ep_layout_dispatch_packed[_fp8]: the checks of ep_layout_packed and ep_dispatch_packed[_fp8].
int check_layout_dispatch_packed(const ep_shape_t *shape, int32_t alignment, int32_t rows,
                                 const uint16_t *x, const int32_t *topk_idx, const int32_t *slot,
                                 const int32_t *expert_count, const int32_t *packed_offset,
                                 const int32_t *stats, const char *fn, int h_multiple)
{
    const std::string f(fn);
    if (int rc = check_layout_args(shape, topk_idx, slot, expert_count, packed_offset, stats, fn))
        return rc;
    if (int rc = check_rows(shape, fn, h_multiple)) return rc;
    if (alignment < 1) return fail(EP_ERR_INVALID, f + ": alignment must be >= 1");
    if ((int64_t)shape->E * ((int64_t)shape->C + alignment - 1) > INT32_MAX)
        return fail(EP_ERR_UNSUPPORTED, f + ": E*(C + alignment - 1) exceeds INT32_MAX");
    if (rows < 0) return fail(EP_ERR_INVALID, f + ": rows must be >= 0");
    if (shape->T > 0 && !x) return fail(EP_ERR_INVALID, f + ": NULL required pointer");
    if (!aligned(x, 16)) return fail(EP_ERR_ALIGN, f + ": x must be 16-byte aligned");
    return EP_OK;
}

}  // namespace

int ep_layout_dispatch_packed(const ep_shape_t *shape, int32_t alignment, int32_t rows,
                              const uint16_t *x, const int32_t *topk_idx, int32_t *slot,
                              int32_t *expert_count, int32_t *packed_offset, int32_t *rank_count,
                              int32_t *rank_offset, int32_t *stats, uint16_t *recv,
                              hipStream_t stream)
{
    const char *fn = "ep_layout_dispatch_packed";
    if (int rc = check_layout_dispatch_packed(shape, alignment, rows, x, topk_idx, slot,
                                              expert_count, packed_offset, stats, fn, 8))
        return rc;
    if (shape->T > 0 && !recv) return fail(EP_ERR_INVALID, "ep_layout_dispatch_packed: NULL required pointer");
    if (!aligned(recv, 16))
        return fail(EP_ERR_ALIGN, "ep_layout_dispatch_packed: recv must be 16-byte aligned");
    ep::LayoutOut o{slot, expert_count, packed_offset, rank_count, rank_offset, stats};
    o.offset_end = packed_offset + shape->E;
    o.align = alignment;
    return hip_status(ep::launch_layout_dispatch_packed_bf16(*shape, x, topk_idx, o, rows, recv,
                                                             stream),
                      fn);
}

int ep_layout_dispatch_packed_fp8(const ep_shape_t *shape, int32_t alignment, int32_t rows,
                                  const uint16_t *x, const int32_t *topk_idx, int32_t *slot,
                                  int32_t *expert_count, int32_t *packed_offset,
                                  int32_t *rank_count, int32_t *rank_offset, int32_t *stats,
                                  uint8_t *recv_q, float *recv_scale, hipStream_t stream)
{
    const char *fn = "ep_layout_dispatch_packed_fp8";
    if (int rc = check_layout_dispatch_packed(shape, alignment, rows, x, topk_idx, slot,
                                              expert_count, packed_offset, stats, fn,
                                              EP_FP8_BLOCK))
        return rc;
    if (shape->T > 0 && (!recv_q || !recv_scale))
        return fail(EP_ERR_INVALID, "ep_layout_dispatch_packed_fp8: NULL required pointer");
    if (!aligned(recv_q, 16) || !aligned(recv_scale, 4))
        return fail(EP_ERR_ALIGN, "ep_layout_dispatch_packed_fp8: recv_q must be 16-byte aligned, "
                                  "recv_scale 4-byte aligned");
    ep::LayoutOut o{slot, expert_count, packed_offset, rank_count, rank_offset, stats};
    o.offset_end = packed_offset + shape->E;
    o.align = alignment;
    return hip_status(ep::launch_layout_dispatch_packed_fp8(*shape, x, topk_idx, o, rows, recv_q,
                                                            recv_scale, stream),
                      fn);
}

int ep_dispatch_packed(const ep_shape_t *shape, int32_t rows, const uint16_t *x,
                       const int32_t *topk_idx, const int32_t *slot,
                       const int32_t *packed_offset, uint16_t *recv, hipStream_t stream)
{
    const char *fn = "ep_dispatch_packed";
    if (int rc = check_packed(shape, rows, packed_offset, fn, 8)) return rc;
    if (shape->T == 0) return hip_status(hipSuccess, fn);
    if (!x || !topk_idx || !slot || !recv) return fail(EP_ERR_INVALID, "ep_dispatch_packed: NULL required pointer");
    if (!aligned(x, 16) || !aligned(recv, 16))
        return fail(EP_ERR_ALIGN, "ep_dispatch_packed: x and recv must be 16-byte aligned");
    return hip_status(ep::launch_dispatch_bf16(*shape, x, topk_idx, slot, recv, stream,
                                               ep::RowMap{packed_offset, rows}),
                      fn);
}

int ep_dispatch_packed_fp8(const ep_shape_t *shape, int32_t rows, const uint16_t *x,
                           const int32_t *topk_idx, const int32_t *slot,
                           const int32_t *packed_offset, uint8_t *recv_q, float *recv_scale,
                           hipStream_t stream)
{
    const char *fn = "ep_dispatch_packed_fp8";
    if (int rc = check_packed(shape, rows, packed_offset, fn, EP_FP8_BLOCK)) return rc;
    if (shape->T == 0) return hip_status(hipSuccess, fn);
    if (!x || !topk_idx || !slot || !recv_q || !recv_scale)
        return fail(EP_ERR_INVALID, "ep_dispatch_packed_fp8: NULL required pointer");
    if (!aligned(x, 16) || !aligned(recv_q, 16) || !aligned(recv_scale, 4))
        return fail(EP_ERR_ALIGN, "ep_dispatch_packed_fp8: x and recv_q must be 16-byte aligned, "
                                  "recv_scale 4-byte aligned");
    return hip_status(ep::launch_dispatch_fp8(*shape, x, topk_idx, slot, recv_q, recv_scale,
                                              stream, ep::RowMap{packed_offset, rows}),
                      fn);
}

int ep_combine_packed(const ep_shape_t *shape, int32_t rows, const uint16_t *y,
                      const int32_t *topk_idx, const int32_t *slot, const int32_t *packed_offset,
                      const float *topk_w, uint16_t *out, hipStream_t stream)
{
    const char *fn = "ep_combine_packed";
    if (int rc = check_packed(shape, rows, packed_offset, fn, 8)) return rc;
    if (shape->T == 0) return hip_status(hipSuccess, fn);
    if (!y || !topk_idx || !slot || !topk_w || !out)
        return fail(EP_ERR_INVALID, "ep_combine_packed: NULL required pointer");
    if (!aligned(y, 16) || !aligned(out, 16))
        return fail(EP_ERR_ALIGN, "ep_combine_packed: y and out must be 16-byte aligned");
    return hip_status(ep::launch_combine(*shape, y, topk_idx, slot, topk_w, out, stream,
                                         ep::RowMap{packed_offset, rows}),
                      fn);
}

namespace {

// Checks shared by the experts' FP8 products: `n` output channels (a multiple of `n_multiple`), for
// each of which an expert has `weight_rows` rows of H channels.
int check_product(const ep_shape_t *shape, int32_t n, int n_multiple, const char *n_name,
                  int weight_rows, const uint8_t *q, const float *scale, const int32_t *expert_count,
                  const uint8_t *w_q, const float *w_scale, const void *out, const char *fn)
{
    const std::string f(fn);
    if (int rc = check_shape(shape, fn)) return rc;
    if (n < 1) return fail(EP_ERR_INVALID, f + ": need " + n_name + " >= 1");
    if (shape->E > EP_MAX_EXPERTS) return fail(EP_ERR_UNSUPPORTED, f + ": E exceeds EP_MAX_EXPERTS");
    if (shape->H % EP_FP8_BLOCK != 0)
        return fail(EP_ERR_UNSUPPORTED, f + ": H must be a multiple of 128");
    if (n % n_multiple != 0)
        return fail(EP_ERR_UNSUPPORTED, f + ": " + n_name + " must be a multiple of " +
                                            std::to_string(n_multiple));
    // lane offsets inside one expert's weights and inside one tile of rows are 32 bits wide
    if ((int64_t)n * weight_rows * shape->H >= int64_t(1) << 30 || shape->H >= 1 << 23)
        return fail(EP_ERR_UNSUPPORTED, f + ": an expert's weights exceed 2^30 elements");
    const bool empty = (int64_t)shape->T * shape->K == 0;
    if (!empty && (!q || !scale || !expert_count || !w_q || !w_scale || !out))
        return fail(EP_ERR_INVALID, f + ": NULL required pointer");
    if (!aligned(q, 16) || !aligned(w_q, 16) || !aligned(out, 16))
        return fail(EP_ERR_ALIGN, f + ": the row buffers and w_q must be 16-byte aligned");
    if (!aligned(scale, 4) || !aligned(expert_count, 4) || !aligned(w_scale, 4))
        return fail(EP_ERR_ALIGN, f + ": scales and counts must be 4-byte aligned");
    return EP_OK;
}

int check_packed_rows(const ep_shape_t *shape, int32_t rows, const int32_t *packed_offset,
                      const char *fn)
{
    const std::string f(fn);
    if (rows < 0) return fail(EP_ERR_INVALID, f + ": need rows >= 0");
    if ((int64_t)shape->T * shape->K > 0 && !packed_offset)
        return fail(EP_ERR_INVALID, f + ": NULL required pointer");
    if (!aligned(packed_offset, 4))
        return fail(EP_ERR_ALIGN, f + ": packed_offset must be 4-byte aligned");
    return EP_OK;
}

ep::ExpertProduct product(const ep_shape_t *s, int32_t n, const uint8_t *q, const float *scale,
                          const int32_t *count, const uint8_t *w_q, const float *w_scale)
{
    ep::ExpertProduct p{};
    p.q = q;
    p.scale = scale;
    p.count = count;
    p.w_q = w_q;
    p.w_scale = w_scale;
    p.E = s->E;
    p.C = s->C;
    p.H = s->H;
    p.n = n;
    p.pairs = s->T * s->K;
    return p;
}

}  // namespace

int ep_expert_gemm_fp8(const ep_shape_t *shape, int32_t N, const uint8_t *recv_q,
                       const float *recv_scale, const int32_t *expert_count, const uint8_t *w_q,
                       const float *w_scale, uint16_t *y, hipStream_t stream)
{
    const char *fn = "ep_expert_gemm_fp8";
    if (int rc = check_product(shape, N, 8, "N", 1, recv_q, recv_scale, expert_count, w_q, w_scale, y,
                               fn))
        return rc;
    ep::ExpertProduct p = product(shape, N, recv_q, recv_scale, expert_count, w_q, w_scale);
    p.y = y;
    return hip_status(ep::launch_expert_gemm_fp8(p, stream), fn);
}

int ep_expert_gemm_fp8_packed(const ep_shape_t *shape, int32_t rows, int32_t N,
                              const uint8_t *recv_q, const float *recv_scale,
                              const int32_t *expert_count, const int32_t *packed_offset,
                              const uint8_t *w_q, const float *w_scale, uint16_t *y,
                              hipStream_t stream)
{
    const char *fn = "ep_expert_gemm_fp8_packed";
    if (int rc = check_product(shape, N, 8, "N", 1, recv_q, recv_scale, expert_count, w_q, w_scale, y,
                               fn))
        return rc;
    if (int rc = check_packed_rows(shape, rows, packed_offset, fn)) return rc;
    ep::ExpertProduct p = product(shape, N, recv_q, recv_scale, expert_count, w_q, w_scale);
    p.offset = packed_offset;
    p.rows = p.C = rows;
    p.y = y;
    return hip_status(ep::launch_expert_gemm_fp8(p, stream), fn);
}

int ep_expert_swiglu_fp8(const ep_shape_t *shape, int32_t I, const uint8_t *recv_q,
                         const float *recv_scale, const int32_t *expert_count,
                         const uint8_t *w_q, const float *w_scale, uint8_t *h_q, float *h_scale,
                         hipStream_t stream)
{
    const char *fn = "ep_expert_swiglu_fp8";
    if (int rc = check_product(shape, I, EP_FP8_BLOCK, "I", 2, recv_q, recv_scale, expert_count, w_q,
                               w_scale, h_q, fn))
        return rc;
    if ((int64_t)shape->T * shape->K > 0 && !h_scale)
        return fail(EP_ERR_INVALID, std::string(fn) + ": NULL required pointer");
    if (!aligned(h_scale, 4))
        return fail(EP_ERR_ALIGN, std::string(fn) + ": scales and counts must be 4-byte aligned");
    ep::ExpertProduct p = product(shape, 2 * I, recv_q, recv_scale, expert_count, w_q, w_scale);
    p.h_q = h_q;
    p.h_scale = h_scale;
    return hip_status(ep::launch_expert_swiglu_fp8(p, stream), fn);
}

int ep_expert_swiglu_fp8_packed(const ep_shape_t *shape, int32_t rows, int32_t I,
                                const uint8_t *recv_q, const float *recv_scale,
                                const int32_t *expert_count, const int32_t *packed_offset,
                                const uint8_t *w_q, const float *w_scale, uint8_t *h_q,
                                float *h_scale, hipStream_t stream)
{
    const char *fn = "ep_expert_swiglu_fp8_packed";
    if (int rc = check_product(shape, I, EP_FP8_BLOCK, "I", 2, recv_q, recv_scale, expert_count, w_q,
                               w_scale, h_q, fn))
        return rc;
    if (int rc = check_packed_rows(shape, rows, packed_offset, fn)) return rc;
    if ((int64_t)shape->T * shape->K > 0 && !h_scale)
        return fail(EP_ERR_INVALID, std::string(fn) + ": NULL required pointer");
    if (!aligned(h_scale, 4))
        return fail(EP_ERR_ALIGN, std::string(fn) + ": scales and counts must be 4-byte aligned");
    ep::ExpertProduct p = product(shape, 2 * I, recv_q, recv_scale, expert_count, w_q, w_scale);
    p.offset = packed_offset;
    p.rows = p.C = rows;
    p.h_q = h_q;
    p.h_scale = h_scale;
    return hip_status(ep::launch_expert_swiglu_fp8(p, stream), fn);
}

size_t ep_moe_layer_workspace_bytes(const ep_shape_t *shape, int32_t I)
{
    if (!shape || shape->T < 0 || shape->E < 1 || shape->K < 1 || shape->H < 1 || I < 1 ||
        (int64_t)shape->T * shape->K > INT32_MAX)
        return 0;
    if (shape->H > 1 << 29 || I > 1 << 29) return 0;     // no call takes them; the sum stays below 2^64
    return ep::moe_workspace_bytes((size_t)shape->T * shape->K, I, shape->H);
}

namespace {

int moe_layer(const ep_shape_t *shape, int32_t I, ep::MoeLayer p, bool fp8, void *workspace,
              size_t workspace_bytes, hipStream_t stream, const char *fn)
{
    const std::string f(fn);
    if (int rc = check_shape(shape, fn)) return rc;
    if (I < 1) return fail(EP_ERR_INVALID, f + ": need I >= 1");
    if (shape->E > EP_MAX_EXPERTS) return fail(EP_ERR_UNSUPPORTED, f + ": E exceeds EP_MAX_EXPERTS");
    if ((int64_t)shape->T * shape->K > EP_MOE_MAX_PAIRS)
        return fail(EP_ERR_UNSUPPORTED, f + ": T*K exceeds EP_MOE_MAX_PAIRS");
    const int step = fp8 ? 128 : 64;
    if (shape->H % step != 0 || I % step != 0)
        return fail(EP_ERR_UNSUPPORTED, f + ": H and I must be multiples of " +
                                            std::to_string(step));
    // byte offsets inside one expert's weights are 32 bits wide
    if ((int64_t)2 * I * shape->H > (int64_t)1 << 29)
        return fail(EP_ERR_UNSUPPORTED, f + ": 2*I*H exceeds 2^29");
    if ((int64_t)shape->T * shape->H > (int64_t)1 << 30 ||
        (int64_t)shape->T * shape->K * I > (int64_t)1 << 29)
        return fail(EP_ERR_UNSUPPORTED, f + ": T*H exceeds 2^30 or T*K*I 2^29");
    if (shape->T == 0) return hip_status(hipSuccess, fn);
    if (!p.x || !p.idx || !p.topk_w || !p.w13 || !p.w2 || !p.out ||
        (fp8 && (!p.w13_scale || !p.w2_scale)))
        return fail(EP_ERR_INVALID, f + ": NULL required pointer");
    if (!aligned(p.x, 16) || !aligned(p.w13, 16) || !aligned(p.w2, 16) || !aligned(p.out, 16))
        return fail(EP_ERR_ALIGN, f + ": x, the weights and out must be 16-byte aligned");
    if (!aligned(p.idx, 4) || !aligned(p.topk_w, 4) || !aligned(p.w13_scale, 4) ||
        !aligned(p.w2_scale, 4))
        return fail(EP_ERR_ALIGN, f + ": ids, weights and scales must be 4-byte aligned");
    const size_t need = ep_moe_layer_workspace_bytes(shape, I);
    if (!workspace) return fail(EP_ERR_INVALID, f + ": workspace is NULL");
    if (workspace_bytes < need)
        return fail(EP_ERR_INVALID, f + ": workspace_bytes " + std::to_string(workspace_bytes) +
                                        " below the " + std::to_string(need) +
                                        " this shape needs");
    if (!aligned(workspace, 16))
        return fail(EP_ERR_ALIGN, f + ": workspace must be 16-byte aligned");
    p.T = shape->T;
    p.E = shape->E;
    p.K = shape->K;
    p.H = shape->H;
    p.I = I;
    const int pairs = shape->T * shape->K;
    p.h = static_cast<uint16_t *>(workspace);
    if (pairs > ep::kMoeSmallPairs) {
        p.y = reinterpret_cast<float *>(p.h + (size_t)2 * pairs * I);
        p.named = reinterpret_cast<int32_t *>(p.y + (size_t)pairs * shape->H);
        p.order = p.named + 4 + (size_t)4 * pairs;
    }
    return hip_status(ep::launch_moe_layer(p, fp8, stream), fn);
}

}  // namespace

int ep_moe_layer(const ep_shape_t *shape, int32_t I, const uint16_t *x, const int32_t *topk_idx,
                 const float *topk_w, const uint16_t *w13, const uint16_t *w2, uint16_t *out,
                 void *workspace, size_t workspace_bytes, hipStream_t stream)
{
    ep::MoeLayer p{};
    p.x = x;
    p.idx = topk_idx;
    p.topk_w = topk_w;
    p.w13 = w13;
    p.w2 = w2;
    p.out = out;
    return moe_layer(shape, I, p, false, workspace, workspace_bytes, stream, "ep_moe_layer");
}

int ep_moe_layer_fp8(const ep_shape_t *shape, int32_t I, const uint16_t *x,
                     const int32_t *topk_idx, const float *topk_w, const uint8_t *w13_q,
                     const float *w13_scale, const uint8_t *w2_q, const float *w2_scale,
                     uint16_t *out, void *workspace, size_t workspace_bytes, hipStream_t stream)
{
    ep::MoeLayer p{};
    p.x = x;
    p.idx = topk_idx;
    p.topk_w = topk_w;
    p.w13 = w13_q;
    p.w13_scale = w13_scale;
    p.w2 = w2_q;
    p.w2_scale = w2_scale;
    p.out = out;
    return moe_layer(shape, I, p, true, workspace, workspace_bytes, stream, "ep_moe_layer_fp8");
}

namespace {

constexpr int32_t kLinearGradMostRows = 1 << 21;    // half the chunks of rows that grid.y holds

// Widths and weights of the bf16 products: rows in 16-byte chunks; lane offsets inside one matrix and
// inside one tile of rows are 32 bits wide.
bool whole_chunks(int64_t H, int64_t N) { return H % 8 == 0 && N % 8 == 0; }

bool widths_fit(int64_t H, int64_t N, int64_t weights)
{
    return H < 1 << 20 && N < 1 << 20 && weights < int64_t(1) << 30;
}

int check_widths(int64_t H, int64_t N, const char *n_name, int64_t weights, const char *fn)
{
    const std::string f(fn);
    if (N < 1) return fail(EP_ERR_INVALID, f + ": need " + n_name + " >= 1");
    if (!whole_chunks(H, N))
        return fail(EP_ERR_UNSUPPORTED, f + ": H and " + n_name + " must be multiples of 8");
    if (!widths_fit(H, N, weights))
        return fail(EP_ERR_UNSUPPORTED, f + ": a width reaches 2^20, or a weight matrix 2^30 elements");
    return EP_OK;
}

// Checks shared by the experts' bf16 products: `n` channels beside H, n * halves rows or columns of an
// expert's weights; `extra` is a third row buffer. A packed buffer may have no rows, and be NULL.
int check_bf16_product(const ep_shape_t *shape, int32_t n, int halves, const char *n_name,
                       const void *x, const void *w, const int32_t *expert_count, const void *extra,
                       const void *out, const char *fn, bool rows = true)
{
    const std::string f(fn);
    if (int rc = check_shape(shape, fn)) return rc;
    if (shape->E > EP_MAX_EXPERTS) return fail(EP_ERR_UNSUPPORTED, f + ": E exceeds EP_MAX_EXPERTS");
    if (int rc = check_widths(shape->H, (int64_t)n * halves, n_name, (int64_t)n * halves * shape->H, fn))
        return rc;
    if (n % 8 != 0)
        return fail(EP_ERR_UNSUPPORTED, f + ": H and " + n_name + " must be multiples of 8");
    if (shape->T > 0 && rows && (!x || !w || !expert_count || !out))
        return fail(EP_ERR_INVALID, f + ": NULL required pointer");
    if (!aligned(x, 16) || !aligned(w, 16) || !aligned(extra, 16) || !aligned(out, 16))
        return fail(EP_ERR_ALIGN, f + ": row buffers, weights and outputs must be 16-byte aligned");
    if (!aligned(expert_count, 4))
        return fail(EP_ERR_ALIGN, f + ": expert_count must be 4-byte aligned");
    return EP_OK;
}

ep::Product bf16_product(const ep_shape_t *s, const uint16_t *x, const uint16_t *w,
                         const int32_t *count, int k, int n, void *out)
{
    ep::Product p{};
    p.x = x;
    p.w = w;
    p.count = count;
    p.E = s->E;
    p.C = s->C;
    p.k = k;
    p.n = n;
    p.pairs = s->T * s->K;
    p.out = out;
    return p;
}

// The packed form of a product.
void pack(ep::Product &p, const int32_t *packed_offset, int32_t rows)
{
    p.offset = packed_offset;
    p.rows = p.C = rows;
    if (rows == 0) p.pairs = 0;
}

int expert_wgrad(const ep_shape_t *shape, int32_t N, const uint16_t *dy, const uint16_t *recv,
                 const int32_t *expert_count, const int32_t *packed_offset, bool packed, int32_t rows,
                 bool f32, int32_t accumulate, void *dw, hipStream_t stream, const char *fn)
{
    if (int rc = check_bf16_product(shape, N, 1, "N", dy, recv, expert_count, nullptr, dw, fn,
                                    !packed || rows != 0))
        return rc;
    if (packed)
        if (int rc = check_packed_rows(shape, rows, packed_offset, fn)) return rc;
    if (!dw) return fail(EP_ERR_INVALID, std::string(fn) + ": NULL required pointer");
    ep::Product p = bf16_product(shape, dy, recv, expert_count, 0, shape->H, dw);
    p.m = N;
    p.accumulate = accumulate != 0;
    if (packed) pack(p, packed_offset, rows);
    return hip_status(ep::launch_expert_wgrad(p, f32, stream), fn);
}

}  // namespace

int ep_expert_gemm(const ep_shape_t *shape, int32_t N, const uint16_t *recv,
                   const int32_t *expert_count, const uint16_t *w, uint16_t *y, hipStream_t stream)
{
    const char *fn = "ep_expert_gemm";
    if (int rc = check_bf16_product(shape, N, 1, "N", recv, w, expert_count, nullptr, y, fn)) return rc;
    return hip_status(
        ep::launch_expert_gemm(bf16_product(shape, recv, w, expert_count, shape->H, N, y), stream), fn);
}

int ep_expert_gemm_packed(const ep_shape_t *shape, int32_t rows, int32_t N, const uint16_t *recv,
                          const int32_t *expert_count, const int32_t *packed_offset,
                          const uint16_t *w, uint16_t *y, hipStream_t stream)
{
    const char *fn = "ep_expert_gemm_packed";
    if (int rc = check_bf16_product(shape, N, 1, "N", recv, w, expert_count, nullptr, y, fn, rows != 0)) return rc;
    if (int rc = check_packed_rows(shape, rows, packed_offset, fn)) return rc;
    ep::Product p = bf16_product(shape, recv, w, expert_count, shape->H, N, y);
    pack(p, packed_offset, rows);
    return hip_status(ep::launch_expert_gemm(p, stream), fn);
}

int ep_expert_swiglu(const ep_shape_t *shape, int32_t I, const uint16_t *recv,
                     const int32_t *expert_count, const uint16_t *w13, uint16_t *gu, uint16_t *h,
                     hipStream_t stream)
{
    const char *fn = "ep_expert_swiglu";
    if (int rc = check_bf16_product(shape, I, 2, "I", recv, w13, expert_count, gu, h, fn)) return rc;
    ep::Product p = bf16_product(shape, recv, w13, expert_count, shape->H, 2 * I, h);
    p.out2 = gu;
    return hip_status(ep::launch_expert_swiglu(p, stream), fn);
}

int ep_expert_swiglu_packed(const ep_shape_t *shape, int32_t rows, int32_t I, const uint16_t *recv,
                            const int32_t *expert_count, const int32_t *packed_offset,
                            const uint16_t *w13, uint16_t *gu, uint16_t *h, hipStream_t stream)
{
    const char *fn = "ep_expert_swiglu_packed";
    if (int rc = check_bf16_product(shape, I, 2, "I", recv, w13, expert_count, gu, h, fn, rows != 0)) return rc;
    if (int rc = check_packed_rows(shape, rows, packed_offset, fn)) return rc;
    ep::Product p = bf16_product(shape, recv, w13, expert_count, shape->H, 2 * I, h);
    p.out2 = gu;
    pack(p, packed_offset, rows);
    return hip_status(ep::launch_expert_swiglu(p, stream), fn);
}

int ep_expert_gemm_dgrad(const ep_shape_t *shape, int32_t N, const uint16_t *dy,
                         const int32_t *expert_count, const uint16_t *w, uint16_t *dx,
                         hipStream_t stream)
{
    const char *fn = "ep_expert_gemm_dgrad";
    if (int rc = check_bf16_product(shape, N, 1, "N", dy, w, expert_count, nullptr, dx, fn)) return rc;
    return hip_status(
        ep::launch_expert_dgrad(bf16_product(shape, dy, w, expert_count, N, shape->H, dx), stream), fn);
}

int ep_expert_gemm_dgrad_packed(const ep_shape_t *shape, int32_t rows, int32_t N, const uint16_t *dy,
                                const int32_t *expert_count, const int32_t *packed_offset,
                                const uint16_t *w, uint16_t *dx, hipStream_t stream)
{
    const char *fn = "ep_expert_gemm_dgrad_packed";
    if (int rc = check_bf16_product(shape, N, 1, "N", dy, w, expert_count, nullptr, dx, fn, rows != 0)) return rc;
    if (int rc = check_packed_rows(shape, rows, packed_offset, fn)) return rc;
    ep::Product p = bf16_product(shape, dy, w, expert_count, N, shape->H, dx);
    pack(p, packed_offset, rows);
    return hip_status(ep::launch_expert_dgrad(p, stream), fn);
}

int ep_expert_swiglu_dgrad(const ep_shape_t *shape, int32_t I, const uint16_t *dy,
                           const int32_t *expert_count, const uint16_t *w2, const uint16_t *gu,
                           uint16_t *dgu, hipStream_t stream)
{
    const char *fn = "ep_expert_swiglu_dgrad";
    if (int rc = check_bf16_product(shape, I, 1, "I", dy, w2, expert_count, gu, dgu, fn)) return rc;
    if (shape->T > 0 && !gu) return fail(EP_ERR_INVALID, std::string(fn) + ": NULL required pointer");
    ep::Product p = bf16_product(shape, dy, w2, expert_count, shape->H, I, dgu);
    p.in = gu;
    return hip_status(ep::launch_expert_swiglu_dgrad(p, stream), fn);
}

int ep_expert_swiglu_dgrad_packed(const ep_shape_t *shape, int32_t rows, int32_t I,
                                  const uint16_t *dy, const int32_t *expert_count,
                                  const int32_t *packed_offset, const uint16_t *w2,
                                  const uint16_t *gu, uint16_t *dgu, hipStream_t stream)
{
    const char *fn = "ep_expert_swiglu_dgrad_packed";
    if (int rc = check_bf16_product(shape, I, 1, "I", dy, w2, expert_count, gu, dgu, fn, rows != 0)) return rc;
    if (shape->T > 0 && rows != 0 && !gu) return fail(EP_ERR_INVALID, std::string(fn) + ": NULL required pointer");
    if (int rc = check_packed_rows(shape, rows, packed_offset, fn)) return rc;
    ep::Product p = bf16_product(shape, dy, w2, expert_count, shape->H, I, dgu);
    p.in = gu;
    pack(p, packed_offset, rows);
    return hip_status(ep::launch_expert_swiglu_dgrad(p, stream), fn);
}

int ep_expert_gemm_wgrad(const ep_shape_t *shape, int32_t N, const uint16_t *dy, const uint16_t *recv,
                         const int32_t *expert_count, uint16_t *dw, hipStream_t stream)
{
    return expert_wgrad(shape, N, dy, recv, expert_count, nullptr, false, 0, false, 0, dw, stream,
                        "ep_expert_gemm_wgrad");
}

int ep_expert_gemm_wgrad_packed(const ep_shape_t *shape, int32_t rows, int32_t N, const uint16_t *dy,
                                const uint16_t *recv, const int32_t *expert_count,
                                const int32_t *packed_offset, uint16_t *dw, hipStream_t stream)
{
    return expert_wgrad(shape, N, dy, recv, expert_count, packed_offset, true, rows, false, 0, dw, stream,
                        "ep_expert_gemm_wgrad_packed");
}

int ep_expert_gemm_wgrad_f32(const ep_shape_t *shape, int32_t N, int32_t accumulate,
                             const uint16_t *dy, const uint16_t *recv, const int32_t *expert_count,
                             float *dw, hipStream_t stream)
{
    return expert_wgrad(shape, N, dy, recv, expert_count, nullptr, false, 0, true, accumulate, dw, stream,
                        "ep_expert_gemm_wgrad_f32");
}

int ep_expert_gemm_wgrad_f32_packed(const ep_shape_t *shape, int32_t rows, int32_t N,
                                    int32_t accumulate, const uint16_t *dy, const uint16_t *recv,
                                    const int32_t *expert_count, const int32_t *packed_offset,
                                    float *dw, hipStream_t stream)
{
    return expert_wgrad(shape, N, dy, recv, expert_count, packed_offset, true, rows, true, accumulate, dw,
                        stream, "ep_expert_gemm_wgrad_f32_packed");
}

namespace {

int combine_grad(const ep_shape_t *shape, const uint16_t *dout, const uint16_t *y,
                 const int32_t *topk_idx, const int32_t *slot, const float *topk_w, uint16_t *dy,
                 float *dtopk_w, ep::RowMap map, hipStream_t stream, const char *fn)
{
    const std::string f(fn);
    const bool rows = !map.offset || map.rows != 0;
    if (shape->T > 0 && (!dout || !topk_idx || !slot || !topk_w || !dtopk_w || (rows && (!y || !dy))))
        return fail(EP_ERR_INVALID, f + ": NULL required pointer");
    if (!aligned(dout, 16) || !aligned(y, 16) || !aligned(dy, 16))
        return fail(EP_ERR_ALIGN, f + ": dout, y and dy must be 16-byte aligned");
    if (!aligned(topk_idx, 4) || !aligned(slot, 4) || !aligned(topk_w, 4) || !aligned(dtopk_w, 4))
        return fail(EP_ERR_ALIGN, f + ": ids, slots and weights must be 4-byte aligned");
    return hip_status(ep::launch_combine_grad(*shape, dout, y, topk_idx, slot, topk_w, dy, dtopk_w,
                                              stream, map),
                      fn);
}

}  // namespace

int ep_combine_grad(const ep_shape_t *shape, const uint16_t *dout, const uint16_t *y,
                    const int32_t *topk_idx, const int32_t *slot, const float *topk_w, uint16_t *dy,
                    float *dtopk_w, hipStream_t stream)
{
    const char *fn = "ep_combine_grad";
    if (int rc = check_shape(shape, fn)) return rc;
    if (int rc = check_rows(shape, fn, 8)) return rc;
    return combine_grad(shape, dout, y, topk_idx, slot, topk_w, dy, dtopk_w, ep::RowMap(), stream, fn);
}

int ep_combine_grad_packed(const ep_shape_t *shape, int32_t rows, const uint16_t *dout,
                           const uint16_t *y, const int32_t *topk_idx, const int32_t *slot,
                           const int32_t *packed_offset, const float *topk_w, uint16_t *dy,
                           float *dtopk_w, hipStream_t stream)
{
    const char *fn = "ep_combine_grad_packed";
    if (int rc = check_packed(shape, rows, packed_offset, fn, 8)) return rc;
    return combine_grad(shape, dout, y, topk_idx, slot, topk_w, dy, dtopk_w,
                        ep::RowMap{packed_offset, rows}, stream, fn);
}

namespace {

int check_linear(const ep_shape_t *shape, int32_t N, int32_t act, const char *fn)
{
    ep::launch_log().n = 0;
    const std::string f(fn);
    if (!shape) return fail(EP_ERR_INVALID, f + ": shape is NULL");
    if (shape->T < 0 || shape->H < 1) return fail(EP_ERR_INVALID, f + ": need T >= 0 and H >= 1");
    if (int rc = check_widths(shape->H, N, "N", (int64_t)N * shape->H, fn)) return rc;
    if (act < EP_ACT_NONE || act > EP_ACT_GELU)
        return fail(EP_ERR_INVALID, f + ": act is no EP_ACT_ value");
    return EP_OK;
}

// A product over the T rows of dense matrices.
ep::Product dense(const ep_shape_t *s, const uint16_t *x, const uint16_t *w, int k, int n, void *out)
{
    const ep_shape_t rows{s->T, s->H, 1, 1, s->T, 1};      // the caller's E, K, C and R may be anything
    return bf16_product(&rows, x, w, nullptr, k, n, out);
}

}  // namespace

int ep_linear(const ep_shape_t *shape, int32_t N, int32_t act, const uint16_t *x, const uint16_t *w,
              const uint16_t *bias, const uint16_t *residual, uint16_t *pre, uint16_t *out,
              hipStream_t stream)
{
    const char *fn = "ep_linear";
    if (int rc = check_linear(shape, N, act, fn)) return rc;
    if (shape->T > 0 && (!x || !w || !out))
        return fail(EP_ERR_INVALID, std::string(fn) + ": NULL required pointer");
    for (const void *q : {(const void *)x, (const void *)w, (const void *)bias, (const void *)residual,
                          (const void *)pre, (const void *)out})
        if (!aligned(q, 16)) return fail(EP_ERR_ALIGN, std::string(fn) + ": arrays must be 16-byte aligned");
    ep::Product p = dense(shape, x, w, shape->H, N, out);
    p.out2 = pre;
    p.in = residual;
    p.bias = bias;
    p.act = act;
    return hip_status(ep::launch_linear(p, stream), fn);
}

size_t ep_linear_grad_workspace_bytes(const ep_shape_t *shape, int32_t N, int32_t act)
{
    if (!shape || shape->T < 0 || shape->T > kLinearGradMostRows || shape->H < 1 || N < 1 ||
        act < EP_ACT_NONE || act > EP_ACT_GELU)
        return 0;
    if (!whole_chunks(shape->H, N) || !widths_fit(shape->H, N, (int64_t)N * shape->H)) return 0;
    const size_t T = shape->T, chunks = (T + ep::kLinearGradRows - 1) / ep::kLinearGradRows;
    return (size_t)N * (4 * chunks + (act == EP_ACT_NONE ? 0 : 2 * T));
}

int ep_linear_grad(const ep_shape_t *shape, int32_t N, int32_t act, const uint16_t *dout,
                   const uint16_t *pre, const uint16_t *x, const uint16_t *w, uint16_t *dx,
                   uint16_t *dw, float *dbias, void *workspace, size_t workspace_bytes,
                   hipStream_t stream)
{
    const char *fn = "ep_linear_grad";
    const std::string f(fn);
    if (int rc = check_linear(shape, N, act, fn)) return rc;
    if (shape->T > kLinearGradMostRows) return fail(EP_ERR_UNSUPPORTED, f + ": T exceeds 2^21");
    const bool some = shape->T > 0;
    if ((some && (!dout || !x || !w || !dx || (act != EP_ACT_NONE && !pre))) || !dw || !dbias)
        return fail(EP_ERR_INVALID, f + ": NULL required pointer");
    for (const void *q : {(const void *)dout, (const void *)pre, (const void *)x, (const void *)w,
                          (const void *)dx, (const void *)dw, (const void *)workspace})
        if (!aligned(q, 16)) return fail(EP_ERR_ALIGN, f + ": arrays must be 16-byte aligned");
    if (!aligned(dbias, 4)) return fail(EP_ERR_ALIGN, f + ": dbias must be 4-byte aligned");
    const size_t need = ep_linear_grad_workspace_bytes(shape, N, act);
    if (need && !workspace) return fail(EP_ERR_INVALID, f + ": workspace is NULL");
    if (workspace_bytes < need)
        return fail(EP_ERR_INVALID, f + ": workspace_bytes " + std::to_string(workspace_bytes) +
                                        " below the " + std::to_string(need) + " this shape needs");
    // dz first: its T*N values are a multiple of 16 bytes
    uint16_t *dz = act == EP_ACT_NONE ? nullptr : static_cast<uint16_t *>(workspace);
    float *part = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) +
                                            (dz ? (size_t)2 * shape->T * N : 0));
    hipError_t e = ep::launch_act_grad(dout, pre, dz, part, dbias, shape->T, N, act, stream);
    const uint16_t *g = dz ? dz : dout;
    if (e == hipSuccess) e = ep::launch_expert_dgrad(dense(shape, g, w, N, shape->H, dx), stream);
    if (e == hipSuccess) {
        ep::Product p = dense(shape, g, x, 0, shape->H, dw);
        p.m = N;
        e = ep::launch_expert_wgrad(p, false, stream);
    }
    return hip_status(e, fn);
}

int ep_check_e4m3_conversion(uint32_t first_pattern, uint32_t count, uint32_t *mismatches,
                             uint32_t *first_mismatch, hipStream_t stream)
{
    ep::launch_log().n = 0;
    if (!mismatches || !first_mismatch)
        return fail(EP_ERR_INVALID, "ep_check_e4m3_conversion: NULL required pointer");
    if ((uint64_t)first_pattern + count > (1ull << 32))
        return fail(EP_ERR_INVALID,
                    "ep_check_e4m3_conversion: first_pattern + count exceeds 2^32");
    if (!aligned(mismatches, 4) || !aligned(first_mismatch, 4))
        return fail(EP_ERR_ALIGN, "ep_check_e4m3_conversion: outputs must be 4-byte aligned");
    return hip_status(ep::launch_check_e4m3(first_pattern, count, mismatches, first_mismatch,
                                            stream),
                      "ep_check_e4m3_conversion");
}

int ep_last_launches(ep_launch_record_t *records, int capacity)
{
    const ep::LaunchLog &log = ep::launch_log();
    const int n = log.n < ep::kLaunchLogCap ? log.n : ep::kLaunchLogCap;
    for (int k = 0; records && k < n && k < capacity; ++k) {
        const ep::LaunchEntry &e = log.e[k];
        ep_launch_record_t &r = records[k];
        const char *name = hipKernelNameRefByPtr(e.kernel, nullptr);
        r.kernel = name ? name : "";
        r.grid_x = e.grid.x;
        r.grid_y = e.grid.y;
        r.grid_z = e.grid.z;
        r.block_x = e.block.x;
        r.block_y = e.block.y;
        r.block_z = e.block.z;
        r.dynamic_lds_bytes = (uint32_t)e.shmem;
        hipFuncAttributes a{};
        if (hipFuncGetAttributes(&a, e.kernel) == hipSuccess) {
            r.static_lds_bytes = (uint32_t)a.sharedSizeBytes;
            r.vgprs = a.numRegs;
            r.private_bytes = (uint32_t)a.localSizeBytes;
            r.max_threads_per_block = a.maxThreadsPerBlock;
        } else {
            r.static_lds_bytes = 0;
            r.vgprs = -1;
            r.private_bytes = 0;
            r.max_threads_per_block = -1;
        }
    }
    return log.n;
}

const char *ep_error_string(int code)
{
    switch (code) {
    case EP_OK: return "EP_OK: success";
    case EP_ERR_INVALID: return "EP_ERR_INVALID: invalid shape or NULL pointer";
    case EP_ERR_ALIGN: return "EP_ERR_ALIGN: buffer not aligned";
    case EP_ERR_UNSUPPORTED: return "EP_ERR_UNSUPPORTED: shape not supported by the kernels";
    case EP_ERR_HIP: return "EP_ERR_HIP: HIP runtime error";
    default: return "unknown ep error code";
    }
}

const char *ep_last_error(void) { return g_last_error.c_str(); }

const char *ep_version(void)
{
    static const std::string v = [] {
        char buf[96];
        snprintf(buf, sizeof buf, "libep_mi355x %s (gfx950; HIP %d.%d.%d)", EP_VERSION_STRING,
                 HIP_VERSION_MAJOR, HIP_VERSION_MINOR, HIP_VERSION_PATCH);
        return std::string(buf);
    }();
    return v.c_str();
}

}  // extern "C"
