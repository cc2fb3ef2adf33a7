"""GB300 (sm_103a) implementation of TACO's fused FP8 compression of
tensor-parallel intermediate tensors ("TACO: Efficient Communication
Compression of Intermediate Tensors for Scalable Tensor-Parallel LLM
Training", Algorithm 1; Sections 4.2-4.4).

    packed = compress(x_bf16, block=128)            # Eqs. 5-10, one fused kernel
    y = decompress(packed, rows, hidden, block=128)  # Eqs. 11-13, one fused kernel
    r = reduce_shards([p0, ..., pP-1], rows, hidden, block=128)  # two-shot local reduction

Every call also takes variant= ("ash_ds", "hadamard_ds", "ds_only",
"ash_only") and code= ("e4m3", "e5m2", "int8") for the paper's ablations.

Training operators next to the codec (layer norm, GELU, 8-bit checkpoints of
activations and the gradients that read them):

    r = layernorm(x, weight, bias, residual=None, checkpoint=True)
    g = layernorm_backward(dy, r.rstd, weight, packed=r.packed)
    r = gelu(x, bias)
    g = gelu_backward(dy, r.packed, bias_dtype=torch.float32)
    dw = weight_grad(dy, packed, hidden)

and those of a gated feed-forward block behind an RMS norm:

    r = rmsnorm(x, weight, residual=None, checkpoint=True)
    g = rmsnorm_backward(dy, r.rstd, weight, packed=r.packed)
    r = gated_linear(x, weight, activation="silu", checkpoint=True)
    g = gated_linear_backward(dy, r.packed, weight)

The kernels live in libtaco_gb300.so (C ABI: include/taco.h); this package
only marshals arguments.  Build the library with
`python -m fp8_compression_tensor_gb300.build`.
"""
from ._binding import (CODES, LIBRARY_PATH, MAX_SHARDS, STATUS, SUPPORTED_BLOCKS, VARIANTS,  # noqa: F401
                       TacoError, compress, compressed_bytes, decompress, device_status, load_library, raw_call,
                       reduce_shards, selftest_encode_bits)
from ._gated import (ACTIVATIONS, GatedLinear, GatedLinearGrads, RmsNorm, RmsNormGrads, gated_linear,  # noqa: F401
                     gated_linear_backward, rmsnorm, rmsnorm_backward)
from ._training import (Gelu, GeluGrads, LayerNorm, LayerNormGrads, gelu, gelu_backward, layernorm,  # noqa: F401
                        layernorm_backward, weight_grad)

__all__ = ["compress", "decompress", "reduce_shards", "compressed_bytes", "device_status", "load_library",
           "TacoError", "LIBRARY_PATH", "MAX_SHARDS", "SUPPORTED_BLOCKS", "STATUS", "VARIANTS", "CODES",
           "raw_call", "selftest_encode_bits", "layernorm", "layernorm_backward", "gelu", "gelu_backward", "weight_grad",
           "LayerNorm", "LayerNormGrads", "Gelu", "GeluGrads", "rmsnorm", "rmsnorm_backward", "gated_linear", "gated_linear_backward",
           "RmsNorm", "RmsNormGrads", "GatedLinear", "GatedLinearGrads", "ACTIVATIONS"]
