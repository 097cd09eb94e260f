"""Bad arguments of a call with a stream are refused as those of one without (CPU: nothing is enqueued)."""
import pytest
import torch

import matrix_orthogonalizing_optimizer_step_amd as mu

Z = torch.zeros(2, 2)
STREAMS = [None, 0, type("Stream", (), {"cuda_stream": 0, "device": torch.device("cuda:0")})()]


@pytest.mark.parametrize("stream", STREAMS, ids=["none", "handle", "object"])
@pytest.mark.parametrize("call", [
    lambda s: mu.adamw_step([], [], [], [], 1, 1e-3, stream=s),
    lambda s: mu.adamw_step([Z], [Z], [Z], [Z], 1, 1e-3, stream=s),
    lambda s: mu.adamw_step([None], [Z], [Z], [Z], 1, 1e-3, stream=s),
    lambda s: mu.adamw8_step([], mu.AdamW8State.zeros([]), [], 1, 1e-3, stream=s),
    lambda s: mu.mx4_quantize([], stream=s),
    lambda s: mu.mx4_quantize(Z, stream=s),
    lambda s: mu.mx4_dequantize(mu.MX4([], [], 4), stream=s),
    lambda s: mu.fp8_quantize([], stream=s),
    lambda s: mu.fp8_quantize([Z], stream=s),
    lambda s: mu.fp8_quantize(None, stream=s),
    lambda s: mu.fp8_dequantize(mu.FP8([], [], 4), stream=s),
    lambda s: mu.fp8_matmul(mu.FP8([], [], 4), mu.FP8([], [], 4), stream=s),
    lambda s: mu.fp8_grouped_matmul(mu.FP8([None], [None], 4), mu.FP8([], [], 4), Z, stream=s),
    lambda s: mu.expert_balance([[1.0]], Z, 1.0, stream=s),
    lambda s: mu.expert_balance(Z, Z.long(), 1.0, stream=s),
])
def test_value_error(call, stream):
    with pytest.raises(ValueError):
        call(stream)
