"""af_weights_quantize_w4 on a stream that is being captured: refused where it
would allocate or free (which would end the capture), recorded where the copy is there."""
import pytest
import torch

import diffusion_transformer_denoising_auraflow_b200 as af
from helpers import af_config, draw_weights, tiny_config, upload

pytestmark = pytest.mark.gpu
UNSUPPORTED = 3


def _pack():
    cfg = tiny_config()
    w = af.Weights(af_config(cfg, dtype=0))
    upload(w, draw_weights(cfg, 891))
    return w


def test_refused_where_it_allocates_or_frees():
    w = _pack()
    x = torch.zeros(8, device="cuda")
    for before, group in ((0, 64), (32, 64), (32, 0)):
        w.quantize_w4(before)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            x += 1
            with pytest.raises(af.AFError) as e:
                w.quantize_w4(group)
            assert e.value.status == UNSUPPORTED
            x += 1
        x.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.all(x == 2)
        w.quantize_w4(group)              # outside it is as ever


def test_recorded_where_the_copy_is_there():
    w = _pack()
    w.quantize_w4(64)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        w.quantize_w4(64)
    g.replay()
    torch.cuda.synchronize()
