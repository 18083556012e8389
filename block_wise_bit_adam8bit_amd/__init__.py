"""block_wise_bit_adam8bit_amd: block-wise dynamic-tree 8-bit Adam for MI355X.

The compute lives in libqopt.so (HIP kernels for gfx950 behind the C ABI of
include/qopt.h, include/qopt_embedding.h, include/qopt_fp8.h, include/qopt_fp4.h,
include/qopt_muon.h, include/qopt_norm.h); this package is its thin Python binding plus torch
optimizers, the Stable Embedding module, layer normalisation and linear layers whose products
run in 8-bit or 4-bit floating point.
Importing it loads the library and fails with ImportError if it is not built.
"""

from ._lib import (  # noqa: F401
    LIB, LIB_PATH, QOPT_BLOCK, QoptError, status_string,
    QOPT_OK, QOPT_EINVAL, QOPT_EUNSUPPORTED, QOPT_EALIGN, QOPT_ELAUNCH, QOPT_EINTERNAL,
    QOPT_ENOSPACE,
    QOPT_CB_SIGNED, QOPT_CB_UNSIGNED, QOPT_F32, QOPT_BF16,
)
from .functional import (  # noqa: F401
    SIGNED, UNSIGNED, nblocks, codebook, codebook_bytes, qopt_codebook_build,
    qopt_quantize_blockwise, qopt_dequantize_blockwise, qopt_adam8bit_step,
    qopt_adam8bit_launch_count, qopt_adam8bit_traffic_probe, qopt_quantize_blockwise_multi,
    qopt_dequantize_blockwise_multi, make_tensor_array, qopt_pattern_probe,
    qopt_pattern_probe_names, AdamWPlan, qopt_adamw8bit_plan, qopt_adamw32bit_plan,
    qopt_adamw8bit_step, qopt_adamw32bit_step,
)
from .checkpoint import (  # noqa: F401
    compress_moments, decompress_moments, compress_moments_multi, decompress_moments_multi,
)
from .optim import Adam8bit, AdamW  # noqa: F401
from .embedding import (  # noqa: F401
    StableEmbedding, StableEmbeddingFunction, qopt_embedding_xavier_init,
    qopt_stable_embedding_forward, qopt_stable_embedding_backward,
)
from .fp8 import (  # noqa: F401
    Fp8Linear, Fp8LinearFunction, Fp8Matrix, fp8_linear, qopt_fp8_linear, qopt_fp8_matmul,
    qopt_fp8_quantize,
)
from .fp4 import (  # noqa: F401
    Fp4Linear, Fp4LinearFunction, Fp4Matrix, fp4_linear, qopt_fp4_dequantize, qopt_fp4_linear,
    qopt_fp4_matmul, qopt_fp4_quantize,
)
from .muon import (  # noqa: F401
    Muon, MuonPlan, qopt_muon32bit_plan, qopt_muon32bit_step, qopt_muon8bit_plan,
    qopt_muon8bit_step, qopt_orthogonalize,
)
from .norm import (  # noqa: F401
    LayerNorm, LayerNormFunction, layer_norm, qopt_layer_norm_backward, qopt_layer_norm_forward,
)

__version__ = "0.1.0"
