// Host-only stand-ins for the kernel side of the selective state space layer's
// operators (ssm_internal.h): they enqueue nothing and count the calls that got
// past the argument checks.
#include "ssm_internal.h"

int g_ssm_enqueued = 0;

namespace ssm {

hipError_t enqueue_conv(const Conv&, hipStream_t) { return ++g_ssm_enqueued, hipSuccess; }
size_t conv_bwd_workspace_bytes(const Conv&) { return 256; }
hipError_t enqueue_conv_bwd(const Conv&, void*, hipStream_t) { return ++g_ssm_enqueued, hipSuccess; }
hipError_t enqueue_scan(const Scan&, hipStream_t) { return ++g_ssm_enqueued, hipSuccess; }
size_t scan_bwd_workspace_bytes(const Scan&) { return 256; }
hipError_t enqueue_scan_bwd(const Scan&, void*, hipStream_t) { return ++g_ssm_enqueued, hipSuccess; }
hipError_t enqueue_block_norm(const BlockNorm&, hipStream_t) { return ++g_ssm_enqueued, hipSuccess; }
size_t block_norm_bwd_workspace_bytes(const BlockNorm&) { return 256; }
hipError_t enqueue_block_norm_bwd(const BlockNorm&, void*, hipStream_t) { return ++g_ssm_enqueued, hipSuccess; }

}  // namespace ssm
