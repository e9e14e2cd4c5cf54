// Launch entry points of the operators of pdn_block.h, called by the host layer
// after argument validation.  Not a public header.
#pragma once
#include <hip/hip_runtime.h>
#include <type_traits>

#include "kernels.h"
#include "pages.h"
#include "pdn_block.h"

namespace pdn {

// Dropout, residual, norm and 8-bit output (add_norm.hip).
hipError_t launch_add_norm(const pdn_add_norm_args& a, hipStream_t stream);
size_t add_norm_bwd_workspace_bytes(const pdn_add_norm_bwd_args& a);
hipError_t launch_add_norm_bwd(const pdn_add_norm_bwd_args& a, hipStream_t stream);

// Attention forward (attn_fwd.hip, the paged one included), its gradient
// (attn_bwd.hip) and the writes into a paged cache (cache.hip).
// Those that end in _fits: whether the launches of such a call keep to 2^32 threads.
bool attn_fits(const pdn_attn_args& a);  // forward and backward
bool attn_paged_fits(const pdn_attn_paged_args& a);
size_t attn_fwd_workspace_bytes(const pdn_attn_args& a);
hipError_t launch_attn_fwd(const pdn_attn_args& a, hipStream_t stream);
size_t attn_bwd_workspace_bytes(const pdn_attn_bwd_args& a);
hipError_t launch_attn_bwd(const pdn_attn_bwd_args& a, hipStream_t stream);
size_t attn_paged_workspace_bytes(const pdn_attn_paged_args& a);
hipError_t launch_attn_paged(const pdn_attn_paged_args& a, hipStream_t stream);
PageMap page_map(const pdn_cache& c);
hipError_t launch_cache_append(const pdn_cache_append_args& a, hipStream_t stream);

}  // namespace pdn
