"""Chunked gated delta-rule forward (KDA / Gated DeltaNet) for MI355X (gfx950).

The forward runs in hand-written HIP kernels behind the C interface of
include/chunk_dr.h (libchunkdr.so); this package is its thin Python binding.  Beside it stand the
norms of a block's boundary, page tables, and latent attention (blocks.py, latent.py).
"""
from .ops import (chunk_dr_fwd, PreparedForward, load_library, workspace_bytes, make_problem, check,  # noqa: F401
                  STAGE_INTRA, STAGE_CHAIN, STAGE_OUTPUT, STAGE_ALL, fused_recurrent_fwd, PreparedRecurrent,
                  chunk_dr_bwd, PreparedBackward, bwd_workspace_bytes,
                  BWD_PREP, BWD_CHAINS, BWD_LOCAL, BWD_ALL, segment_map, merge_states,
                  chunk_dr_fwd_noalloc, NOALLOC_SCRATCH_BYTES, check_cu_seqlens)
from .blocks import block_norm_fwd, block_norm_bwd, build_page_tables, PageTables  # noqa: F401
from .latent import (latent_cache_write, latent_decode_fwd, latent_decode_workspace_bytes,  # noqa: F401
                     latent_attn_fwd, latent_attn_bwd)
