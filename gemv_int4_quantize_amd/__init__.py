"""MI355X-native quantized linear operators: weight-only int4 (W4A16) quantize-and-pack and
mixed-precision matmul, the 8-bit integer (W8A8) and microscaled 4-bit (MXFP4) products and
their gradients, layers of experts on MXFP4 weights, and the scores of tokens under the logits
that they give.

The compute lives in ``libw4a16.so`` (hand-written HIP for gfx950, C ABI in
``include/w4a16.h``, ``include/w8a8.h`` and ``include/mxfp4.h``); this package is its PyTorch binding.
"""

from ._lib import LIB_PATH, W4Desc, W4Error, lib  # noqa: F401
from .ops import (  # noqa: F401
    QuantizedWeight,
    dequantize,
    deserialize,
    load,
    empty_quantized,
    kernel_for,
    meta_shape,
    mm,
    mm_plan,
    mm_split,
    mode_id,
    quantize_fused,
    quantize_pack,
    quantize_pack_into,
    save,
    serialize,
)
from .int8 import (  # noqa: F401
    Int8Rows,
    int8_kernel_for,
    mm_int8,
    mm_int8_split,
    mm_int8_t,
    quantize_int8,
)
from .mxfp4 import (  # noqa: F401
    MXFP4Rows,
    dequantize_mxfp4,
    mm_mxfp4,
    mm_mxfp4_split,
    mm_mxfp4_t,
    moe_mxfp4,
    mxfp4_kernel_for,
    quantize_mxfp4,
)
from .layer import (  # noqa: F401
    MXFP4Linear,
    MXFP4MoE,
    W4A16Linear,
    W8A8Linear,
    mxfp4_linear,
    w4a16_linear,
    w8a8_linear,
)
from .scores import TokenLogprobs, token_logprobs, token_logprobs_grad  # noqa: F401

__version__ = "0.1.0"
