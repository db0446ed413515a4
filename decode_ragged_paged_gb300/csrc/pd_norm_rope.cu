// pd_norm_rope.cu -- launches of the norm and rotation (pd_norm_rope.cuh), and its
// kernels for positions with one axis.
#include "pd_norm_rope.cuh"

namespace pd {

// Elements of a lane's run: the widest (at most 16 bytes) that divides the
// halves of the head and of its rotated part, keeps every row aligned, and
// gives a head to at most 32 lanes; 0 if there is none.
int32_t norm_rope_vec(const NormRopeParams& p, int32_t elem_size, uintptr_t addresses) {
  const int64_t strides = p.q_stride | p.k_stride | p.v_stride | p.q_out_stride | p.k_out_stride;
  for (int v = 16 / elem_size; v >= 2; v >>= 1) {
    if (p.head_dim % (2 * v) != 0 || p.rope_dim % (2 * v) != 0 || strides % v != 0) continue;
    if (addresses % (uintptr_t)(v * elem_size) != 0) continue;
    return p.head_dim / (2 * v) <= 32 ? v : 0;
  }
  return 0;
}

int launch_norm_rope(NormRopeParams& p, int32_t elem_size, int32_t vec, cudaStream_t stream) {
  const int units = p.head_dim / (2 * vec);
  p.lanes = 1;
  while (p.lanes < units) p.lanes <<= 1;
  p.heads_per_group = 32 / p.lanes;
  // groups of q heads, of k heads, and (with a slot map) of v heads
  p.q_groups = (p.hq + p.heads_per_group - 1) / p.heads_per_group;
  p.kv_groups = (p.hkv + p.heads_per_group - 1) / p.heads_per_group;
  p.groups = p.q_groups + (p.slot_map != nullptr ? 2 : 1) * p.kv_groups;
  p.inv_dim = 1.0f / (float)p.head_dim;
  p.staged = vec * elem_size == 16;
  // A warp takes as many of a token's head groups as leave every SM its resident
  // warps (more would reuse its cosines further, but leave SMs without work), and
  // no more than a stage holds.
  const int64_t resident = (int64_t)device_sm_count() * 2;  // CTAs
  int64_t blocks = (resident * (kNrThreads / 32) + p.tokens - 1) / p.tokens;
  if (p.staged && blocks < (p.groups + kNrStageGroups - 1) / kNrStageGroups)
    blocks = (p.groups + kNrStageGroups - 1) / kNrStageGroups;
  if (blocks > p.groups) blocks = p.groups;
  p.groups_per_block = (int32_t)((p.groups + blocks - 1) / blocks);
  p.blocks = (p.groups + p.groups_per_block - 1) / p.groups_per_block;
  const int64_t items = (int64_t)p.tokens * p.blocks;
  int64_t grid = (items * 32 + kNrThreads - 1) / kNrThreads;
  if (grid > resident) grid = resident;
  last_kernel() = "norm_rope_kernel";
  profile_begin(stream);
  const cudaError_t e = p.num_axes > 0 ? launch_norm_rope_axes(p, elem_size, vec, (unsigned)grid, stream)
                                       : launch_norm_rope_form<false>(p, elem_size, vec, (unsigned)grid, stream);
  profile_end(stream);
  return e == cudaSuccess ? PD_OK : PD_ERR_CUDA;
}

}  // namespace pd
