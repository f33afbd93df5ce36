"""MI355X (gfx950) QLoRA NF4 linear layer: HIP kernels behind a C ABI
(include/qlora_nf4.h) and a thin ctypes binding (``binding``)."""
from .binding import (CODEBOOK_INT4, CODEBOOK_NF4, GradList, PackedInt8, PackedNF4, QloraError,  # noqa: F401
                      dequantize, dequantize_int8, dropout_mask, dropout_workspace_bytes, grad_clip, grad_norm,
                      grouped_workspace_bytes, int8_linear_fwd, levels, linear_bwd,
                      linear_bwd_dropout, linear_bwd_grouped, linear_fwd, linear_fwd_dropout, linear_fwd_grouped,
                      load, load_packed, merge, quantize, quantize_int8, requantize, rmsnorm_int8, save_packed,
                      status_string, unmerge, workspace_bytes)
