"""EXL3 decode-row projection for MI355X (gfx950): rot_in and the trellis linear, and
the operators around it: attention of drafted trees over a paged cache, the cache's
append, verification of the drafts and distillation of a drafter; norms and rotation of
queries and keys, attention of whole prompts, and a cache in 4 bits.

The compute runs in libtf_exl3.so (hand-written HIP kernels behind the C ABI in
include/tf_exl3.h); this package only marshals torch tensors and streams into
those calls. Importing it does not touch the GPU; the first call loads the
library and raises if it has not been built.
"""

from ._lib import (  # noqa: F401
    TF_DT_BF16,
    TF_DT_F16,
    TF_DT_F32,
    Exl3Error,
    debug_decode_states,
    calib_copy,
    calib_stream_read,
    debug_decode_tiles,
    debug_linear_split,
    debug_linear_mfma_split,
    header_functions,
    linear,
    linear_plan,
    project,
    project_pass_rows,
    repack_strips,
    load,
    rot_in,
    status_string,
    trellis_bytes,
)
from ._ops import (  # noqa: F401
    cache_append,
    distill,
    distill_grad,
    distill_loss,
    tree_attention,
    verify_chain,
    verify_tree,
)
from ._rows import (  # noqa: F401
    cache_append_q4,
    cache_read_q4,
    norm_rotate,
    prompt_attention,
    q4_row_bytes,
    tree_attention_q4,
)

WIDTHS = (2, 3, 4, 5, 6, 8)
