"""A missing tensor in the 4-bit and residual-norm calls is a TypeError that names it (no GPU needed)."""
import pytest
import torch

import diffusion_transformer_denoising_auraflow_b200 as af

BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8


def z(*shape, dtype=F32):
    return torch.zeros(*shape, dtype=dtype)


X, CODES, SCALES, OUT, ROWS = z(3, 100), z(5, 64, dtype=U8), z(4, 8, dtype=BF), z(3, 5), z(2, 3, 16)
CALLS = [
    (af.linear_w4, dict(x=X, codes=CODES, scales=SCALES, group=32, out=OUT), ("x", "codes", "scales", "out")),
    (af.quantize_rows_w4, dict(w=z(5, 100), group=32, codes=CODES, scales=SCALES), ("w", "codes", "scales")),
    (af.dequantize_rows_w4, dict(codes=CODES, scales=SCALES, group=32, out=z(5, 100)), ("codes", "scales", "out")),
    (af.residual_norm, dict(x=ROWS, branch=ROWS, x_out=ROWS, y=ROWS, eps=1e-6), ("x",)),
    (af.residual_norm_e4m3, dict(x=ROWS, branch=ROWS, x_out=ROWS, y8=z(2, 3, 16, dtype=U8), yscale=z(6), eps=1e-6),
     ("x", "y8", "yscale")),
]


@pytest.mark.parametrize("fn,args,name", [(f, a, n) for f, a, names in CALLS for n in names])
@pytest.mark.parametrize("value", [None, [1.0]])
def test_missing_tensor_is_named(fn, args, name, value):
    with pytest.raises(TypeError, match=f"{name} must be"):
        fn(**{**args, name: value})
