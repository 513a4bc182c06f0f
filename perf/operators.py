"""What the training-step operators beside the attention operator are measured on.

Two families: layer norm with the residual added on the way in (forward,
backward, and both as one training step), and the global gradient norm over a
list of tensors with clipping. `run` computes them in plain torch operations,
or, where `own` is true, with this package's calls.
"""
import math
import random

import torch

own = False  # set from outside: run() makes this package's calls

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
EPS = 1e-5


def listed():
    """The measured cases: layer norm (`op` norm) by direction, and clipping (`op` clip)."""
    norm, clip = dict(op="norm"), dict(op="clip")
    return [
        # a detector decoder's 300 queries, one image: the inference call where latency counts
        dict(norm, name="norm decoder bf16", way="forward", rows=300, cols=256, dtype="bf16", residual=True, total=False, params="bf16"),
        # one token of a wide model being decoded
        dict(norm, name="norm one row fp16", way="forward", rows=1, cols=8192, dtype="fp16", residual=True, total=True, params="fp16"),
        # the Deformable-DETR encoder's tokens, two images of 22,223
        dict(norm, name="norm encoder bf16", way="forward", rows=44446, cols=256, dtype="bf16", residual=True, total=False, params="bf16"),
        # rows of odd length: no row but the first is aligned
        dict(norm, name="norm odd fp16", way="forward", rows=20011, cols=777, dtype="fp16", residual=False, total=False, params="fp32"),
        # the decoder's training step, two images
        dict(norm, name="norm decoder step fp32", way="step", rows=600, cols=256, dtype="fp32", residual=True, total=False, params="fp32"),
        # the encoder's backward pass alone
        dict(norm, name="norm encoder backward bf16", way="backward", rows=44446, cols=256, dtype="bf16", residual=True, total=False, params="bf16"),
        # the Mask2Former pixel decoder's tokens, four images of 21,504, in fp32
        dict(norm, name="norm mask encoder step fp32", way="step", rows=86016, cols=256, dtype="fp32", residual=True, total=False, params="fp32"),
        # a wide pre-norm stack: the sum goes on beside the normalised rows, weights kept in fp32
        dict(norm, name="norm wide step bf16", way="step", rows=8192, cols=4096, dtype="bf16", residual=True, total=True, params="fp32"),
        # the gradients of one attention layer with its norm
        dict(clip, name="clip layer fp32", layout="layer", tensors=10, elements=0, dtype="fp32", out="fp32", kind="2", limit=0.1),
        # the gradients of a whole detector: convolutions, encoder and decoder layers, heads
        dict(clip, name="clip detector fp32", layout="detector", tensors=0, elements=0, dtype="fp32", out="fp32", kind="2", limit=0.1),
        # bf16 gradients of a large model into fp32 master gradients
        dict(clip, name="clip large bf16 to fp32", layout="drawn", tensors=291, elements=300_000_000, dtype="bf16", out="fp32", kind="2", limit=1.0),
        # the largest entry of fp16 gradients, watched for overflow; nothing is clipped
        dict(clip, name="largest entry fp16", layout="drawn", tensors=150, elements=60_000_000, dtype="fp16", out="none", kind="inf", limit=0.0),
    ]


def draw(rng):
    """One more case: sizes spread over their logarithms, odd and ragged ones among them."""
    if rng.random() < 0.6:
        rows = int(math.exp(rng.uniform(0, math.log(90_000))))
        cols = int(math.exp(rng.uniform(math.log(16), math.log(12_000))))
        if rng.random() < 0.5:
            cols = -(-cols // 32) * 32
        rows = max(1, min(rows, 30_000_000 // cols))
        dtype = rng.choice(["fp32", "bf16", "fp16"])
        residual = rng.random() < 0.6
        return dict(op="norm", way=rng.choice(["forward", "backward", "step"]), rows=rows, cols=cols, dtype=dtype, residual=residual,
                    total=residual and rng.random() < 0.4, params=rng.choice([dtype, "fp32"]))
    tensors = int(math.exp(rng.uniform(0, math.log(400))))
    elements = max(40 * tensors, int(math.exp(rng.uniform(math.log(10_000), math.log(200_000_000)))))
    dtype = rng.choice(["fp32", "bf16", "fp16"])
    return dict(op="clip", layout="drawn", tensors=tensors, elements=elements, dtype=dtype, out=rng.choice([dtype, "fp32", "none"]),
                kind=rng.choice(["2", "2", "inf"]), limit=rng.choice([0.1, 1.0, 1e9]))


def sizes_of(case):
    """The element counts of a clip case's tensors."""
    d, bias = 256, 256
    if case["layout"] == "layer":  # offsets, logits, value and output projections (8 heads, 4 levels, 4 points), norm
        return [256 * d, 256, 128 * d, 128, d * d, d, d * d, d, d, d]
    if case["layout"] == "detector":
        conv = []
        for blocks, width, cin in ((3, 64, 64), (4, 128, 256), (6, 256, 512), (3, 512, 1024)):
            for b in range(blocks):
                conv += [(cin if b == 0 else 4 * width) * width, width * width * 9, width * 4 * width]
                conv += [cin * 4 * width] if b == 0 else []
        attention = [256 * d, 256, 128 * d, 128, d * d, d, d * d, d]
        ffn = [1024 * d, 1024, d * 1024, d, d, bias, d, bias]
        head = [91 * d, 91, d * d, d, d * d, d, 4 * d, 4]
        return [64 * 3 * 49] + conv + [512 * d, d, 1024 * d, d, 2048 * d, d, 2048 * d * 9, d] + (attention + ffn) * 6 + \
            ([3 * d * d, 3 * d, d * d, d, d, d] + attention + ffn) * 6 + head * 6 + [4 * d, 300 * 2 * d]
    # a few matrices hold most of the entries, many vectors hold few
    rng = random.Random(case["tensors"] * 1_000_003 + case["elements"])
    share = [math.exp(rng.uniform(-9, 0)) for _ in range(case["tensors"])]
    return [max(1, int(case["elements"] * s / sum(share))) for s in share]


def uniform_rows(case, gen):
    """Activations as a trained stack has them: channels of their own size and offset, a few far larger."""
    rows, cols = case["rows"], case["cols"]
    size = torch.randn(cols, device="cuda", generator=gen).mul_(0.5).exp_()
    size[:: max(1, cols // 3)] *= 8
    x = torch.randn(rows, cols, device="cuda", generator=gen)
    return (x * size + 0.3 * torch.randn(cols, device="cuda", generator=gen)).to(DTYPES[case["dtype"]])


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    state = dict(case=dict(case))
    if case["op"] == "norm":
        rows, cols, dtype, params = case["rows"], case["cols"], DTYPES[case["dtype"]], DTYPES[case["params"]]
        state["x"] = uniform_rows(case, gen)
        state["residual"] = uniform_rows(case, gen) if case["residual"] else None
        state["weight"] = (1 + 0.2 * torch.randn(cols, device="cuda", generator=gen)).to(params)
        state["bias"] = (0.1 * torch.randn(cols, device="cuda", generator=gen)).to(params)
        if case["way"] != "forward":
            state["grad"] = (0.01 * torch.randn(rows, cols, device="cuda", generator=gen)).to(dtype)
            state["grad_total"] = (0.01 * torch.randn(rows, cols, device="cuda", generator=gen)).to(dtype) if case["total"] else None
        if case["way"] == "backward":  # what the forward pass left
            s = state["x"].double() + (state["residual"].double() if case["residual"] else 0)
            state["mean"] = s.mean(-1).float()
            state["rstd"] = (s.var(-1, unbiased=False) + EPS).rsqrt().float()
        if case["way"] == "step":
            state["leaves"] = [state[k].requires_grad_() for k in ("x", "residual", "weight", "bias") if state[k] is not None]
        return state
    sizes, dtype = sizes_of(case), DTYPES[case["dtype"]]
    flat = torch.randn(sum(sizes), device="cuda", generator=gen)
    scale = torch.randn(len(sizes), device="cuda", generator=gen).mul_(1.5).exp_().mul_(0.01)
    state["grads"] = [(g * s).to(dtype) for g, s in zip(flat.split(sizes), scale.unbind())]
    state["flat"] = None
    if case["out"] != "none":  # the clipped gradients, one after another
        state["flat"] = torch.empty(sum(sizes), device="cuda", dtype=DTYPES[case["out"]])
    if own:  # the handle that a training loop keeps over its gradient buffers
        from scale_deformable_attention_msda_gb300 import binding
        state["buffers"] = binding.GradientBuffers(state["grads"], out=None if state["flat"] is None else list(state["flat"].split(sizes)))
    return state


def run(state):
    if own:
        return run_own(state)
    with torch.no_grad():
        return plain_norm(state) if state["case"]["op"] == "norm" else plain_clip(state)


def run_own(state):
    from scale_deformable_attention_msda_gb300 import binding
    case = state["case"]
    if case["op"] == "clip":
        if state["flat"] is None:
            return binding.msda_grad_norm(state["buffers"], norm_type=float(case["kind"]))
        norm = binding.msda_clip_grad_norm(state["buffers"], case["limit"], norm_type=float(case["kind"]))
        return [norm, state["flat"]]
    if case["way"] == "backward":
        grad_x, grad_weight, grad_bias = binding.msda_layer_norm_backward(
            state["grad"], state["x"], state["mean"], state["rstd"], weight=state["weight"],
            residual=state["residual"], grad_sum=state["grad_total"])
        return [grad_x, grad_weight, grad_bias]
    out = binding.layer_norm(state["x"], state["weight"], state["bias"], residual=state["residual"], eps=EPS, return_sum=case["total"])
    outs = list(out) if case["total"] else [out]
    if case["way"] == "forward":
        return outs
    grads = torch.autograd.grad(outs, state["leaves"], [state["grad"], state["grad_total"]][: len(outs)])
    return [o.detach() for o in outs] + [grads[0], grads[-2], grads[-1]]


def plain_norm(state):
    case, dtype, params = state["case"], state["x"].dtype, state["weight"].dtype
    s = state["x"].float()
    if state["residual"] is not None:
        s = s + state["residual"].float()
    weight, outs = state["weight"].float(), []
    if case["way"] == "backward":
        mean, rstd = state["mean"][:, None], state["rstd"][:, None]
        xhat = (s - mean) * rstd
    else:
        mean = s.mean(-1, keepdim=True)
        centred = s - mean
        rstd = 1.0 / torch.sqrt((centred * centred).mean(-1, keepdim=True) + EPS)
        xhat = centred * rstd
        outs = [(xhat * weight + state["bias"].float()).to(dtype)] + ([s.to(dtype)] if case["total"] else [])
    if case["way"] == "forward":
        return outs
    dy = state["grad"].float()
    g = dy * weight
    dx = rstd * (g - g.mean(-1, keepdim=True) - xhat * (g * xhat).mean(-1, keepdim=True))
    if state["grad_total"] is not None:
        dx = dx + state["grad_total"].float()
    return outs + [dx.to(dtype), (dy * xhat).sum(0).to(params), dy.sum(0).to(params)]


def plain_clip(state):
    case = state["case"]
    flat = torch.cat([g.reshape(-1) for g in state["grads"]]).float()
    # squares are summed in 64 bits: hundreds of millions of them
    norm = flat.abs().max() if case["kind"] == "inf" else flat.double().square().sum().sqrt().float()
    if case["out"] == "none":
        return norm
    factor = torch.clamp(case["limit"] / (norm + 1e-6), max=1.0)
    return [norm, (flat * factor).to(DTYPES[case["out"]])]


def work(case):
    if case["op"] == "norm":
        n, e, p = case["rows"] * case["cols"], DTYPES[case["dtype"]].itemsize, DTYPES[case["params"]].itemsize
        reads, writes, params, stats = 1 + case["residual"], 0, 2, 0
        if case["way"] != "backward":
            writes += 1 + case["total"]
        if case["way"] != "forward":
            reads, writes, params = reads + 1 + case["total"], writes + 1, params + 2
        if case["way"] == "backward":
            params, stats = 3, 2
        flops = n * {"forward": 8, "backward": 14, "step": 22}[case["way"]]
        return dict(bytes=n * e * (reads + writes) + case["cols"] * p * params + 4 * stats * case["rows"], flops=flops)
    n = sum(sizes_of(case))
    if case["out"] == "none":
        return dict(bytes=n * DTYPES[case["dtype"]].itemsize, flops=2 * n)
    return dict(bytes=n * (DTYPES[case["dtype"]].itemsize + DTYPES[case["out"]].itemsize), flops=3 * n)


def exact(case, seed):
    """The definitions in 64 bits; gradients by differentiating the definition."""
    state = prepare(case, seed)
    if case["op"] == "clip":
        grads = [g.to(torch.float64) for g in state["grads"]]
        if case["kind"] == "inf":
            norm = torch.stack([g.abs().amax() for g in grads]).amax()
        else:
            norm = torch.stack([torch.dot(g, g) for g in grads]).sum() ** 0.5
        if case["out"] == "none":
            return norm
        total = float(norm) + 1e-6
        return [norm, torch.cat(grads) * (case["limit"] / total if total > case["limit"] else 1.0)]
    leaf = {k: state[k].detach().to(torch.float64).requires_grad_() for k in ("x", "weight", "bias")}
    s = leaf["x"] if state["residual"] is None else leaf["x"] + state["residual"].detach().to(torch.float64)
    variance, mean = torch.var_mean(s, dim=-1, correction=0, keepdim=True)
    y = (s - mean) / (variance + EPS) ** 0.5 * leaf["weight"] + leaf["bias"]
    outs = [y, s] if case["total"] else [y]
    if case["way"] == "forward":
        return [o.detach() for o in outs]
    into = [state["grad"].to(torch.float64)] + ([state["grad_total"].to(torch.float64)] if case["total"] else [])
    grads = torch.autograd.grad(outs, [leaf["x"], leaf["weight"], leaf["bias"]], into)
    return ([] if case["way"] == "backward" else [o.detach() for o in outs]) + list(grads)
