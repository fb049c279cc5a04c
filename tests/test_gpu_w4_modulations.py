"""The model with its modulation weights in 4 bits (af_weights_quantize_w4)
against the oracle with the values those weights stand for.

The quantiser's decisions are the same on both sides, so what is left is the
arithmetic of the paths themselves: the tolerances are theirs (blocks 2e-2 on
the update, the full stack 5e-2, the fp32 model 1e-4).
"""
import numpy as np
import pytest
import torch

import oracle as O
import synth
from helpers import af_config, block_names, draw_weights, tiny_config, to_bf16, to_f32, to_np, upload

pytestmark = pytest.mark.gpu
BLOCK_TOL, STACK_TOL, F32_TOL = 2e-2, 5e-2, 1e-4


@pytest.fixture(scope="module")
def af():
    import diffusion_transformer_denoising_auraflow_b200 as m
    return m


def _with_values(drawn, group):
    """The drawn weights with every modulation linear replaced by its 4-bit values."""
    out = dict(drawn)
    for name, a in drawn.items():
        if ".norm1" in name or name.startswith("norm_out"):
            c, s = O.quantize_rows_w4(a, group)
            out[name] = O.dequantize_rows_w4(c, s, group, a.shape[1])
    return out


def _tiny(af, seed, dtype, group, B=2):
    cfg = tiny_config()
    w = af.Weights(af_config(cfg, dtype=dtype))
    drawn = draw_weights(cfg, seed, dtype="f32" if dtype else "bf16")
    upload(w, drawn)
    w.quantize_w4(group)
    s = af.Scratch(w, B, 64, 8)
    return cfg, w, s, drawn, _with_values(drawn, group)


@pytest.mark.parametrize("dtype,tol,group", [(0, STACK_TOL, 32), (0, STACK_TOL, 64), (1, F32_TOL, 32), (1, F32_TOL, 128)])
def test_tiny_forward(af, dtype, tol, group):
    cfg, w, s, drawn, values = _tiny(af, 881, dtype, group)
    d = "f32" if dtype else "bf16"
    lat = synth.latents(882, (2, 4, 16, 16))
    text = synth.text_embeddings(883, (2, 8, cfg.joint_attention_dim), d)
    t = np.array([0.7, 0.2], np.float32)
    te = to_f32(text) if dtype else to_bf16(text)
    vel = torch.empty(2, 4, 16, 16, device="cuda")
    af.transformer_forward(w, s, to_f32(lat), te, to_f32(t), vel)
    s.sync()
    ref = O.transformer_forward(lat, text, t, values, cfg)
    assert O.rel_l2(to_np(vel), ref) < tol
    if dtype:  # fp32: far nearer to the 4-bit model than the two models are to each other
        other = O.rel_l2(O.transformer_forward(lat, text, t, drawn, cfg), ref)
        assert other > 10 * O.rel_l2(to_np(vel), ref)
    # off again: bit for bit what a pack that never was in 4 bits gives
    w.quantize_w4(0)
    a, b = torch.empty_like(vel), torch.empty_like(vel)
    af.transformer_forward(w, s, to_f32(lat), te, to_f32(t), a)
    w2 = af.Weights(af_config(cfg, dtype=dtype))
    upload(w2, drawn)
    s2 = af.Scratch(w2, 2, 64, 8)
    af.transformer_forward(w2, s2, to_f32(lat), te, to_f32(t), b)
    s2.sync()
    assert torch.equal(a, b)


def test_single_block_real_width(af):
    cfg = O.Config(num_mmdit_layers=0, num_single_dit_layers=1, pos_embed_max_size=64 * 64)
    pre = "single_transformer_blocks.0."
    w = af.Weights(af_config(cfg))
    drawn = draw_weights(cfg, 884, block_names(cfg, "single", 0))
    upload(w, drawn)
    w.quantize_w4(64)
    s = af.Scratch(w, 2, 256, 64)
    x = synth.activations(885, "w4x", (2, 120, 3072))
    temb = synth.conditioning(886, (2, 3072))
    xt = to_bf16(x)
    af.single_block(w, s, 0, xt, to_f32(temb))
    s.sync()
    ref = O.single_block(x, temb, _with_values(drawn, 64), pre, cfg)
    assert O.rel_l2(to_np(xt) - x, ref - x) < BLOCK_TOL


def _storage_floor(x_next, x):
    """A residual stream kept in bf16 is rounded at both gated additions of a
    block, each by at most 2^-8 of the value, so an update is known only to
    2 * 2^-8 |x'| / |x' - x|; at 32 columns with weights of 0.02 the gates are so
    small that this is most of the update."""
    return 2 * 2.0 ** -8 * np.linalg.norm(x_next) / np.linalg.norm(np.asarray(x_next) - x)


@pytest.mark.parametrize("cfg,Ni,Nt", [(tiny_config(), 64, 16),
                                       (O.Config(num_mmdit_layers=1, num_single_dit_layers=0,
                                                 pos_embed_max_size=64 * 64), 96, 24)])
def test_joint_block_with_8_bit_projections(af, cfg, Ni, Nt):
    """4-bit modulations next to the 8-bit projections (their tolerance, 5e-2)."""
    pre = "joint_transformer_blocks.0."
    D = cfg.inner_dim
    w = af.Weights(af_config(cfg))
    drawn = draw_weights(cfg, 887, None if D == 32 else block_names(cfg, "joint", 0))
    upload(w, drawn)
    w.quantize_fp8()
    w.quantize_w4(32)
    s = af.Scratch(w, 2, Ni, Nt)
    img, txt = synth.activations(888, "i", (2, Ni, D)), synth.activations(889, "t", (2, Nt, D))
    temb = synth.conditioning(890, (2, D))
    it, tt = to_bf16(img), to_bf16(txt)
    af.joint_block(w, s, 0, it, tt, to_f32(temb))
    s.sync()
    rt, ri = O.joint_block(img, txt, temb, _with_values(drawn, 32), pre, cfg, fp8=True)
    for got, ref, x in ((it, ri, img), (tt, rt, txt)):
        tol = 5e-2 + (_storage_floor(ref, x) if D == 32 else 0.0)
        assert O.rel_l2(to_np(got) - x, ref - x) < tol


@pytest.mark.parametrize("n", [2, 12])
def test_sampler(af, n):
    """prepare() takes the modulations of all steps (n rows) from the 4-bit
    weights; two steps, with graphs, against the oracle's loop."""
    cfg, w, s, drawn, values = _tiny(af, 891, 0, 32)
    x0 = synth.latents(892, (1, 4, 16, 16))
    text = synth.text_embeddings(893, (2, 8, cfg.joint_attention_dim))
    sig = af.sigma_schedule(n)
    xt, tt = to_f32(x0), to_bf16(text)
    stream = torch.cuda.Stream()
    smp = af.Sampler(w, s, xt, tt, sig, 3.5, use_graphs=True)
    with torch.cuda.stream(stream):
        smp.prepare(stream)
        for i in range(2):
            smp.step(i, stream)
    stream.synchronize()
    s.sync()
    x = x0.astype(np.float64)
    for i in range(2):
        v = O.transformer_forward(np.concatenate([x, x]), text, np.full(2, sig[i]), values, cfg)
        x = O.euler_cfg_step(x, v, 3.5, sig[i], sig[i + 1])
    assert O.rel_l2(to_np(xt) - x0, x - x0) < STACK_TOL
    smp.close()


def test_follows_weight_changes_and_refuses(af):
    cfg, w, s, drawn, _ = _tiny(af, 894, 0, 32)
    x = synth.activations(895, "x", (1, 20, 32))
    temb = to_f32(synth.conditioning(896, (1, 32)))

    def block():
        xt = to_bf16(x)
        af.single_block(w, s, 0, xt, temb)
        s.sync()
        return xt

    before = block()
    name = "single_transformer_blocks.0.norm1.linear.weight"
    w.set(name, to_bf16(2 * drawn[name]))
    assert torch.equal(block(), before)          # the copy is the weights' at the time of the call
    w.quantize_w4(32)
    after = block()
    assert not torch.equal(after, before)
    w.quantize_w4(64)                            # another group: made anew
    w.quantize_w4(32)
    assert torch.equal(block(), after)
    for bad in (16, 1, -32, 256):
        with pytest.raises(af.AFError) as ei:
            w.quantize_w4(bad)
        assert ei.value.status == 3
    assert torch.equal(block(), after)
    assert af.lib.af_weights_quantize_w4(None, 32, None) == 1
