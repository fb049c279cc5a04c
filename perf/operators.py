"""The 4-bit products and fused residual norms, as cases to be timed and compared.

Three operators, in plain elementary torch (own = False) or through the
framework's calls (own = True):

  linear_w4      out = f(x) (s (c - 8))^T + bias: rows of 4-bit codes c with one
                 bf16 scale s per group of `group` columns; f is the identity or
                 SiLU.  The adaLN-Zero modulations of a denoising step.
  quantize_w4    codes and scales of a weight matrix, and the values they stand for.
  residual_norm  u = post(branch) post_weight; x' = x + r g u;
                 y = pre(x') pre_weight (1 + scale) + shift, post and pre each no
                 norm, LayerNorm or RMS norm: what lies between two sub-blocks.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one block's six modulation vectors of the smallest model (width 32): latency
        dict(name="w4 tiny", op="linear_w4", M=1, N=192, K=32, group=32, x="f32", out="f32", silu=True, bias=False),
        # one single block's modulations for the guidance pair
        dict(name="w4 block", op="linear_w4", M=2, N=18432, K=3072, group=64, x="f32", out="f32", silu=True,
             bias=False),
        # every modulation of a denoising step at once, the guidance pair
        dict(name="w4 step", op="linear_w4", M=2, N=743424, K=3072, group=64, x="f32", out="f32", silu=True,
             bias=False),
        # a ragged projection of a few tokens, with a bias
        dict(name="w4 ragged", op="linear_w4", M=7, N=4099, K=2051, group=32, x="bf16", out="bf16", silu=False,
             bias=True),
        # a joint block's modulations for all 25 sampling steps
        dict(name="w4 plan", op="linear_w4", M=25, N=36864, K=3072, group=128, x="f32", out="f32", silu=True,
             bias=False),
        # quantising a small odd weight
        dict(name="q4 odd", op="quantize_w4", N=517, K=1003, group=32, w="f32"),
        # quantising the modulation weights of four blocks
        dict(name="q4 blocks", op="quantize_w4", N=73728, K=3072, group=64, w="bf16"),
        # one token between two sub-blocks: latency
        dict(name="rn token", op="residual_norm", B=1, N=1, D=3072, t="bf16", y="bf16", post="none", pre="layer",
             gate=True, mod=True, post_w=False, pre_w=False, r=1.0),
        # the smallest model in fp32, both norms
        dict(name="rn odd f32", op="residual_norm", B=3, N=77, D=1001, t="f32", y="f32", post="rms", pre="rms",
             gate=False, mod=False, post_w=True, pre_w=True, r=0.5),
        # adaLN-Zero between attention and feed-forward at 1024 x 1024, the guidance pair
        dict(name="rn 1024", op="residual_norm", B=2, N=4360, D=3072, t="bf16", y="bf16", post="none", pre="layer",
             gate=True, mod=True, post_w=False, pre_w=False, r=1.0),
        # the same with 8-bit output and a normalised branch
        dict(name="rn 1024 8-bit", op="residual_norm", B=2, N=4360, D=3072, t="bf16", y="e4m3", post="rms",
             pre="layer", gate=True, mod=True, post_w=True, pre_w=False, r=0.7),
        # 1536 x 1536, norms on both sides of the block
        dict(name="rn 1536", op="residual_norm", B=2, N=9480, D=3072, t="bf16", y="bf16", post="layer", pre="rms",
             gate=True, mod=True, post_w=True, pre_w=True, r=0.7),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["linear_w4", "linear_w4", "quantize_w4", "residual_norm", "residual_norm"])
    if op == "linear_w4":
        M, K = _log(rng, 1, 32), _log(rng, 16, 8192)
        N = min(_log(rng, 1, 200000), 2 * 743424 * 3072 // (M * K))
        x = rng.choice(["bf16", "f32"])
        return dict(op=op, M=M, N=N, K=K, group=rng.choice([32, 64, 128]), x=x, out=rng.choice(["bf16", "f32"]),
                    silu=rng.random() < 0.5, bias=rng.random() < 0.5)
    if op == "quantize_w4":
        K = _log(rng, 1, 8192)
        return dict(op=op, N=min(_log(rng, 1, 70000), 73728 * 3072 // K), K=K, group=rng.choice([32, 64, 128]),
                    w=rng.choice(["bf16", "f32"]))
    B, D = rng.randint(1, 4), _log(rng, 8, 8192)
    t = rng.choice(["bf16", "bf16", "f32"])
    most = 2 * 9480 * 3072 // (1 if t == "bf16" else 2)
    N = max(1, min(_log(rng, 1, 9480), most // (B * D)))
    post = rng.choice(["none", "layer", "rms"])
    return dict(op=op, B=B, N=N, D=D, t=t, y=rng.choice([t, t, "e4m3"]) if t == "bf16" else t, post=post,
                pre=rng.choice(["none", "layer", "rms"]), gate=rng.random() < 0.7, mod=rng.random() < 0.7,
                post_w=post != "none" and rng.random() < 0.5, pre_w=rng.random() < 0.3, r=rng.choice([1.0, 0.7, 0.125]))


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dtype=torch.float32, std=1.0):
        return torch.randn(*shape, device="cuda", dtype=dtype, generator=g).mul_(std)

    s = dict(case)
    if case["op"] == "linear_w4":
        M, N, K, G = case["M"], case["N"], case["K"], case["group"]
        groups = -(-K // G)
        s["xv"] = normal(M, K, dtype=DTYPES[case["x"]])
        # codes of normal weights: a group's largest value lands on +-7; code 8 (zero) behind column K
        q = normal(N, groups * G, dtype=torch.bfloat16, std=2.8).round_().clamp_(-7, 7).add_(8).to(torch.uint8)
        q[:, K:] = 8
        s["codes"] = (q[:, 0::2] | (q[:, 1::2] << 4)).contiguous()
        s["scales"] = normal(groups, -(-N // 8) * 8, std=0.0012).add_(0.008).abs_().to(torch.bfloat16)
        s["biasv"] = normal(N, std=0.1) if case["bias"] else None
        s["outv"] = torch.empty(M, N, device="cuda", dtype=DTYPES[case["out"]])
    elif case["op"] == "quantize_w4":
        N, K, G = case["N"], case["K"], case["group"]
        groups = -(-K // G)
        s["wv"] = normal(N, K, dtype=DTYPES[case["w"]], std=0.02)
        s["codes"] = torch.empty(N, groups * G // 2, device="cuda", dtype=torch.uint8)
        s["scales"] = torch.empty(groups, -(-N // 8) * 8, device="cuda", dtype=torch.bfloat16)
        s["outv"] = torch.empty(N, K, device="cuda", dtype=DTYPES[case["w"]])
    else:
        B, N, D, t = case["B"], case["N"], case["D"], DTYPES[case["t"]]
        s["xv"] = normal(B, N, D, dtype=t, std=2.0)
        s["bv"] = normal(B, N, D, dtype=t)
        # one table of modulation rows per sample, cut into gate, shift and scale
        table = normal(B, 3 * D, std=0.5)
        s["gatev"], s["shiftv"], s["scalev"] = table[:, :D], table[:, D:2 * D], table[:, 2 * D:]
        s["post_wv"] = normal(D, std=0.2).add_(1) if case["post_w"] else None
        s["pre_wv"] = normal(D, std=0.2).add_(1) if case["pre_w"] else None
        s["xo"] = torch.empty(B, N, D, device="cuda", dtype=t)
        if case["y"] == "e4m3":
            s["yv"] = torch.empty(B, N, D, device="cuda", dtype=torch.uint8)
            s["ys"] = torch.empty(B * N, device="cuda")
        else:
            s["yv"] = torch.empty(B, N, D, device="cuda", dtype=t)
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    return {"linear_w4": _linear, "quantize_w4": _quantize, "residual_norm": _residual_norm}[s["op"]](s)


def _linear(s):
    if own:
        import diffusion_transformer_denoising_auraflow_b200 as af
        af.linear_w4(s["xv"], s["codes"], s["scales"], s["group"], s["outv"], silu=s["silu"], bias=s["biasv"])
        return s["outv"]
    N, K, G = s["N"], s["K"], s["group"]
    w = torch.stack([s["codes"] & 15, s["codes"] >> 4], -1).view(N, -1, G).float().sub_(8)
    w.mul_(s["scales"][:, :N].float().t().unsqueeze(-1))
    x = s["xv"].float()
    if s["silu"]:
        x = x / (1 + torch.exp(-x))
    out = x @ w.view(N, -1)[:, :K].t()
    if s["biasv"] is not None:
        out = out + s["biasv"]
    return out.to(s["outv"].dtype)


def _quantize(s):
    if own:
        import diffusion_transformer_denoising_auraflow_b200 as af
        af.quantize_rows_w4(s["wv"], s["group"], s["codes"], s["scales"])
        af.dequantize_rows_w4(s["codes"], s["scales"], s["group"], s["outv"])
        return s["outv"], s["scales"][:, :s["N"]]
    N, K, G = s["N"], s["K"], s["group"]
    w = torch.nn.functional.pad(s["wv"].float(), (0, -K % G)).view(N, -1, G)
    # a tensor as the divisor: division itself, not a product with the reciprocal
    scale = (w.abs().amax(-1) / torch.full((), 7.0, device=w.device)).to(torch.bfloat16)
    d = scale.float().unsqueeze(-1)
    q = torch.where(d > 0, (w / d).round(), 0.0)
    return (q * d).view(N, -1)[:, :K].to(s["outv"].dtype), scale.t()


def _norm(v, kind):
    if kind == "layer":
        v = v - v.mean(-1, keepdim=True)
    if kind != "none":
        v = v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS)
    return v


def _residual_norm(s):
    eight = s["y"] == "e4m3"
    if own:
        import diffusion_transformer_denoising_auraflow_b200 as af
        more = dict(gate=s["gatev"] if s["gate"] else None, shift=s["shiftv"] if s["mod"] else None,
                    scale=s["scalev"] if s["mod"] else None, mod_stride=3 * s["D"], residual_scale=s["r"],
                    post=s["post"], post_weight=s["post_wv"], pre=s["pre"], pre_weight=s["pre_wv"])
        if eight:
            af.residual_norm_e4m3(s["xv"], s["bv"], s["xo"], s["yv"], s["ys"], EPS, **more)
            return s["xo"], s["yv"].view(torch.float8_e4m3fn), s["ys"]
        af.residual_norm(s["xv"], s["bv"], s["xo"], s["yv"], EPS, **more)
        return s["xo"], s["yv"]
    u = _norm(s["bv"].float(), s["post"])
    if s["post_wv"] is not None:
        u = u * s["post_wv"]
    if s["gate"]:
        u = u * s["gatev"].unsqueeze(1)
    x = s["xv"].float() + s["r"] * u
    y = _norm(x, s["pre"])
    if s["pre_wv"] is not None:
        y = y * s["pre_wv"]
    if s["mod"]:
        y = y * (1 + s["scalev"].unsqueeze(1)) + s["shiftv"].unsqueeze(1)
    xo = x.to(s["xo"].dtype)
    if not eight:
        return xo, y.to(s["yv"].dtype)
    # the value a row's code stands for is code * scale
    top = y.abs().amax(-1, keepdim=True)
    codes = (y * torch.where(top > 0, 448 / top, 1.0)).to(torch.float8_e4m3fn)
    return xo, codes, torch.where(top > 0, top / 448, 1.0).view(-1)


# ---------------------------------------------------------------- work and the exact answer
def work(case):
    if case["op"] == "linear_w4":
        M, N, K, G = case["M"], case["N"], case["K"], case["group"]
        e = {"bf16": 2, "f32": 4}
        return {"bytes": N * K / 2 + 2 * N * -(-K // G) + M * K * e[case["x"]] + M * N * e[case["out"]]
                + (4 * N if case["bias"] else 0), "flops": 2 * M * N * K}
    if case["op"] == "quantize_w4":
        N, K, G = case["N"], case["K"], case["group"]
        e = {"bf16": 2, "f32": 4}[case["w"]]
        return {"bytes": 2 * e * N * K + 2 * N * -(-K // G), "flops": 3 * N * K}
    B, N, D = case["B"], case["N"], case["D"]
    e = {"bf16": 2, "f32": 4}[case["t"]]
    y = 1 if case["y"] == "e4m3" else e
    vectors = B * (case["gate"] + 2 * case["mod"]) + case["post_w"] + case["pre_w"]
    return {"bytes": B * N * D * (3 * e + y) + 4 * D * vectors + (4 * B * N if y == 1 else 0),
            "flops": 16 * B * N * D}


def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "linear_w4":
        x = s["xv"].to(f64)
        x = x * torch.sigmoid(x) if case["silu"] else x
        K, G = case["K"], case["group"]
        out = torch.empty(case["M"], case["N"], dtype=f64, device="cuda")
        for n in range(0, case["N"], 16384):  # a part of the rows at a time
            c = s["codes"][n:n + 16384].to(torch.int16)
            w = torch.empty(c.shape[0], 2 * c.shape[1], dtype=f64, device="cuda")
            w[:, 0::2], w[:, 1::2] = (c % 16) - 8, torch.div(c, 16, rounding_mode="floor") - 8
            sc = s["scales"][:, n:n + c.shape[0]].to(f64).repeat_interleave(G, 0).t()
            out[:, n:n + 16384] = torch.matmul(x, (w * sc)[:, :K].t())
        return out if s["biasv"] is None else out + s["biasv"].to(f64)
    if case["op"] == "quantize_w4":
        N, K, G = case["N"], case["K"], case["group"]
        out = torch.empty(N, K, dtype=f64, device="cuda")
        scales = torch.empty(-(-K // G), N, dtype=f64, device="cuda")
        for j in range(scales.shape[0]):  # a group of columns at a time
            w = s["wv"][:, j * G:(j + 1) * G].to(f64)
            # the scale and the codes are whole decisions: a / 7 in 64 bits, rounded to bf16
            sc = (w.abs().max(1).values / torch.tensor(7.0, dtype=f64, device="cuda")).to(torch.bfloat16).to(f64)
            q = torch.round(w / sc.clamp_min(1e-300)[:, None])
            out[:, j * G:(j + 1) * G] = q * sc[:, None]
            scales[j] = sc
        return out, scales
    x, b = s["xv"].to(f64), s["bv"].to(f64)

    def normed(v, kind):
        if kind == "none":
            return v
        var, mean = torch.var_mean(v, -1, keepdim=True, correction=0)
        return (v - mean) / torch.sqrt(var + EPS) if kind == "layer" else v / torch.sqrt(var + mean ** 2 + EPS)

    u = normed(b, case["post"])
    if case["post_w"]:
        u = u * s["post_wv"].to(f64)
    if case["gate"]:
        u = torch.einsum("bnd,bd->bnd", u, s["gatev"].to(f64))
    x = torch.add(x, u, alpha=case["r"])
    y = normed(x, case["pre"])
    if case["pre_w"]:
        y = y * s["pre_wv"].to(f64)
    if case["mod"]:
        y = torch.einsum("bnd,bd->bnd", y, s["scalev"].to(f64) + 1) + s["shiftv"].to(f64)[:, None]
    if case["y"] != "e4m3":
        return x, y
    top = torch.linalg.vector_norm(y, float("inf"), -1)
    top = torch.where(top == 0, 448.0, top)
    return x, y * (448.0 / top)[..., None], top.view(-1) / 448.0
