"""MI355X-native Muon optimizer step: momentum, standard or Gram Newton-Schulz
orthogonalisation and the weight update, in hand-written HIP kernels for
gfx950 behind the C ABI of include/muon.h, with the AdamW step for the other
parameters and the microscaled 4-bit code and product for the updated weights.
This package is the thin binding (``binding``, with the extension module
``_native`` for lists of tensors) and the build script (``_build``)."""
from .binding import (  # noqa: F401
    BF16, F16, F32, GRAM, MX4, STANDARD, AdamW8State, GraspState, MuonError, NSConfig, abi_version, adamw8_step,
    adamw_step, grasp_step, grasp_workspace_size, gram_ns_orthogonalize, grid_dequantize, grid_quantize,
    group8_dequantize, group8_quantize, load_library, mfma_ceiling, muon_step, muon_step_fixed_scratch,
    mx4_dequantize, mx4_matmul, mx4_quantize, mx4_workspace_size, ns_flops, ns_orthogonalize, pointer_array,
    quintic_schedule, trace_collect, trace_enable, workspace, workspace_size,
)
