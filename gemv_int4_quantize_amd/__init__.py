"""MI355X-native quantized linear operators: weight-only int4 (W4A16) quantize-and-pack and
mixed-precision matmul, the 8-bit integer (W8A8) product and its gradient, and the scores
of tokens under the logits that they give.

The compute lives in ``libw4a16.so`` (hand-written HIP for gfx950, C ABI in
``include/w4a16.h`` and ``include/w8a8.h``); this package is its PyTorch binding.
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
from .layer import W4A16Linear, W8A8Linear, w4a16_linear, w8a8_linear  # noqa: F401
from .scores import TokenLogprobs, token_logprobs, token_logprobs_grad  # noqa: F401

__version__ = "0.1.0"
