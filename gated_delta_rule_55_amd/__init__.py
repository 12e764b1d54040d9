"""KDA (Kimi Delta Attention) forward on AMD MI355X: chunked prefill and
recurrent decode, and the short causal conv before them, as hand-written HIP
kernels behind a C ABI (include/kda.h, include/kda_conv.h); linear attention
with a decay per head (include/kda_linear.h) and the norms of a layer around
either (include/kda_norm.h); latent attention over a paged cache, for the layers
between them (include/kda_latent.h)."""
from .kda import (  # noqa: F401
    causal_conv1d_fwd,
    causal_conv1d_update,
    chunk_prefill,
    prefill_workspace_bytes,
    recurrent_decode,
    recurrent_prefill,
    workspace_status,
)
from .latent import (  # noqa: F401
    latent_append,
    latent_decode,
    latent_extend,
    latent_prefill, latent_prefill_workspace_bytes,
    latent_workspace_bytes,
    rotary,
    rotary_frequencies,
)
from .layer import (  # noqa: F401
    block_norm,
    gated_norm,
    linear_decode,
    linear_prefill,
    linear_workspace_bytes,
)
from ._abi import KdaError, LIB_PATH  # noqa: F401
