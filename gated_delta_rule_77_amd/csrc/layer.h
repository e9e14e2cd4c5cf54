// Launch entry points of the operators around the recurrence, called by the
// host layer after argument validation.  Not a public header.
#pragma once
#include <hip/hip_runtime.h>

#include "kernels.h"
#include "pdn_layer.h"

namespace pdn {

// A launch has fewer than 2^32 threads in a dimension.  The functions below that
// end in _fits say whether a call of these sizes keeps to that.
constexpr long kMaxGridThreads = (1L << 32) - 1;

// Norm and rotation of q and k into the recurrence's layout, and the gated
// norm of its output, with their gradients (head_norm.hip).
bool qk_norm_fits(const pdn_qk_norm_args& a);
hipError_t launch_qk_norm(const pdn_qk_norm_args& a, hipStream_t stream);
size_t qk_norm_bwd_workspace_bytes(const pdn_qk_norm_bwd_args& a);
hipError_t launch_qk_norm_bwd(const pdn_qk_norm_bwd_args& a, hipStream_t stream);
bool out_norm_fits(const pdn_out_norm_args& a);
hipError_t launch_out_norm(const pdn_out_norm_args& a, hipStream_t stream);
size_t out_norm_bwd_workspace_bytes(const pdn_out_norm_bwd_args& a);
hipError_t launch_out_norm_bwd(const pdn_out_norm_bwd_args& a, hipStream_t stream);

// The recurrence with a vector state (scan.hip).
bool scan_fits(const pdn_scan_args& a);
size_t scan_fwd_workspace_bytes(const pdn_scan_args& a);
size_t scan_bwd_workspace_bytes(const pdn_scan_bwd_args& a);
hipError_t launch_scan_fwd(const pdn_scan_args& a, hipStream_t stream);
hipError_t launch_scan_bwd(const pdn_scan_bwd_args& a, hipStream_t stream);
hipError_t launch_scan_step(const pdn_scan_step_args& a, hipStream_t stream);

}  // namespace pdn
