"""Float64 CPU oracle for the FLASH GAU forward (test infrastructure only).

Only the test suite, ``__graft_entry__.smoke()`` and the CPU-baseline leg of
``bench.py`` may import this package.  The CUDA library never does, and the
two share no code.
"""

from .flash_gau import (  # noqa: F401
    swish,
    scale_offset,
    relpos_bias,
    chunk_scores,
    chunk_mask,
    layer_norm,
    scale_norm,
    rope,
    rope_toeplitz_bias,
    toeplitz_relpos,
    flash_gau,
    flash_block,
    algorithmic_flops_per_token,
)
from .backward import swish_grad, flash_gau_backward  # noqa: F401,E402
from .decode import DecodeState  # noqa: F401,E402
from .training import (  # noqa: F401,E402
    norm_rows, residual_norm, residual_norm_grad, xent, adamw, adamw_codes, decode_moments,
    encode_moments,
)
from .language import (  # noqa: F401,E402
    buckets_of_offsets, bucket_bias, bucket_bias_grad, checkpoint_codes, checkpoint_values,
    sample_row,
)
