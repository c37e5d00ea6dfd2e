"""B200-native (sm_100a) forward path of the ReLU-gated sparse FFN with TwELL.

    y = (x W_u  (.)  ReLU(x W_g)) W_d

computed as a tcgen05 gate GEMM whose epilogue packs the ReLU gate into TwELL
(Tile-wise ELLPACK), a fused sparse up+down kernel over the active units, and
a dense-row tensor-core path for tiles that overflow the TwELL capacity.

Around it: the layer norm that feeds the FFN and its backward pass, and the
dense FFN's 8-bit integer form (rows quantised to int8, products with a scale
per token and channel).
"""
from .twell import (  # noqa: F401
    CapacityError,
    Int8FFN,
    KernelTrace,
    TwellBuffers,
    TwellError,
    dense_ffn,
    dense_ffn_int8,
    dequantize_rows,
    ffn_fwd,
    gate_pack,
    int8_ffn_weights,
    int8_gated,
    int8_linear,
    last_launch_count,
    layer_norm,
    layer_norm_bwd,
    layer_norm_int8,
    lib,
    quantize_rows,
    read_status,
    sparse_ffn,
)
