"""What attention between queries and keys, and dropout, are measured on.

Two families of a detector decoder's sublayers: attention of queries over keys
(forward, its backward pass, and both as one training step), and dropout from a
counter-based generator with a residual (forward, and a training step). `run`
computes them in plain torch operations, or, where `own` is true, with this
package's calls.
"""
import math

import numpy
import torch

own = False  # set from outside: run() makes this package's calls

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    """The measured cases: attention (`op` attend) by direction, and dropout (`op` drop)."""
    attend = dict(op="attend", mask="none", share=1.0, fused=False)
    drop = dict(op="drop")
    return [
        # a detector decoder's 300 queries among themselves, one image: the inference call where latency counts
        dict(attend, name="attend decoder bf16", way="forward", batch=1, queries=300, keys=300, heads=8, kv_heads=8, dim=32, dtype="bf16"),
        # one query token (a class token, a prompt) over four long feature maps, key heads shared by four query heads
        dict(attend, name="attend one query fp16", way="forward", batch=4, queries=1, keys=16384, heads=16, kv_heads=4, dim=64, dtype="fp16"),
        # the decoder's training step in fp32, two images
        dict(attend, name="attend decoder step fp32", way="step", batch=2, queries=300, keys=300, heads=8, kv_heads=8, dim=32, dtype="fp32"),
        # 900 queries with 200 denoising queries in front, whose groups must not see one another
        dict(attend, name="attend denoising step bf16", way="step", batch=4, queries=1100, keys=1100, heads=8, kv_heads=8, dim=32, dtype="bf16", mask="groups"),
        # 100 mask queries over a 128 x 128 map, each only where its mask was; some masks are empty
        dict(attend, name="attend masked map bf16", way="forward", batch=4, queries=100, keys=16384, heads=8, kv_heads=8, dim=32, dtype="bf16", mask="regions", share=0.3),
        # the backward pass alone of the same over the 64 x 64 map
        dict(attend, name="attend masked map backward fp16", way="backward", batch=4, queries=100, keys=4096, heads=8, kv_heads=8, dim=32, dtype="fp16", mask="regions", share=0.3),
        # a batch of unequal images, padded: odd lengths, q, k and v out of one projection
        dict(attend, name="attend padded step fp16", way="step", batch=6, queries=1333, keys=1333, heads=12, kv_heads=12, dim=64, dtype="fp16", mask="padding", share=0.8, fused=True),
        # a wide dense encoder's training step, key heads shared by four query heads
        dict(attend, name="attend wide step bf16", way="step", batch=2, queries=4096, keys=4096, heads=16, kv_heads=4, dim=128, dtype="bf16"),
        # dropout after the decoder's self-attention, two images of 300 queries, added to the residual stream
        dict(drop, name="dropout decoder bf16", way="forward", rows=600, cols=256, dtype="bf16", residual=True, p=0.1),
        # the same for the encoder's tokens, two images of 22,223, with its gradient
        dict(drop, name="dropout encoder step bf16", way="step", rows=44446, cols=256, dtype="bf16", residual=True, p=0.1),
        # inside a feed-forward block, in fp32
        dict(drop, name="dropout wide step fp32", way="step", rows=44446, cols=1024, dtype="fp32", residual=False, p=0.1),
        # rows of odd length
        dict(drop, name="dropout odd fp16", way="forward", rows=20011, cols=777, dtype="fp16", residual=True, p=0.3),
    ]


def draw(rng):
    """One more case: sizes spread over their logarithms, odd and ragged ones among them."""
    def spread(low, high):
        return int(math.exp(rng.uniform(math.log(low), math.log(high + 1))))

    if rng.random() < 0.3:
        cols = spread(8, 8192)
        rows = max(1, min(spread(1, 90_000), 40_000_000 // cols))
        return dict(op="drop", way=rng.choice(["forward", "step"]), rows=rows, cols=cols, dtype=rng.choice(["fp32", "bf16", "fp16"]),
                    residual=rng.random() < 0.6, p=rng.choice([0.05, 0.1, 0.3, 0.5]))
    mask = rng.choice(["none", "none", "groups", "regions", "padding"])
    dtype = rng.choice(["fp32", "bf16", "bf16", "fp16", "fp16"])
    dim = rng.choice([16, 24, 32, 32, 40, 64, 64, 80, 96, 128])
    kv_heads = rng.choice([1, 2, 3, 4, 8])
    heads = kv_heads * rng.choice([1, 1, 1, 2, 4])
    batch = rng.randint(1, 6)
    kind = rng.random()
    if mask == "groups" or kind < 0.5:
        queries = keys = spread(16, 4096)
    elif kind < 0.7:
        queries, keys = 1, spread(1, 20_000)
    else:
        queries, keys = spread(2, 300), spread(16, 20_000)
    # no more scores than 2^28 (32-bit data: 2^25)
    most = 2 ** 25 if dtype == "fp32" else 2 ** 28
    while batch * heads * queries * keys > most and batch > 1:
        batch -= 1
    while batch * heads * queries * keys > most:
        queries, keys = (queries + 1) // 2, (keys + 1) // 2
    return dict(op="attend", way=rng.choice(["forward", "backward", "step"]), batch=batch, queries=queries, keys=keys, heads=heads, kv_heads=kv_heads,
                dim=dim, dtype=dtype, mask=mask, share=1.0 if mask in ("none", "groups") else rng.choice([0.2, 0.5, 0.8]),
                fused=queries == keys and rng.random() < 0.4)


def denoising_groups(length):
    """How many queries in front denoise, and how many of them make a group."""
    front = length * 2 // 11
    return front, max(1, front // 5)


def make_mask(case, gen):
    """A bool mask that broadcasts to (batch, heads, queries, keys): true where a query may attend."""
    batch, queries, keys = case["batch"], case["queries"], case["keys"]
    if case["mask"] == "none":
        return None
    if case["mask"] == "padding":  # an image's keys end early, the longest image's do not
        ends = torch.rand(batch, device="cuda", generator=gen) * 2 * (1 - case["share"])
        ends = ((1 - ends.clamp(max=0.95)) * keys).ceil().long().clamp(min=1)
        ends[0] = keys
        return (torch.arange(keys, device="cuda") < ends[:, None])[:, None, None, :]
    if case["mask"] == "groups":
        front, size = denoising_groups(queries)
        at = torch.arange(queries, device="cuda")
        group = torch.where(at < front, at // size, -1)
        return (group[None, :] == -1) | (group[:, None] == group[None, :])
    # regions: an interval of the map's rows for each query, one in sixteen of them empty
    width = max(1, int(math.sqrt(keys)))
    high = (keys + width - 1) // width
    middle = torch.rand(batch, queries, 1, device="cuda", generator=gen) * high
    reach = torch.rand(batch, queries, 1, device="cuda", generator=gen) * case["share"] * high
    reach = torch.where(torch.rand(batch, queries, 1, device="cuda", generator=gen) < 1 / 16, -1.0, reach)
    row = torch.arange(keys, device="cuda") // width
    return ((row + 0.5 - middle).abs() <= reach)[:, None]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype = DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    state = dict(case=dict(case))
    if case["op"] == "drop":
        shape = (case["rows"], case["cols"])
        state["x"] = normal(*shape).to(dtype)
        state["residual"] = (2 * normal(*shape)).to(dtype) if case["residual"] else None
        state["grad"] = (0.01 * normal(*shape)).to(dtype) if case["way"] == "step" else None
        # the generator's seed and the number of this draw
        state["counter"] = torch.randint(-2 ** 62, 2 ** 62, (2,), device="cuda", generator=gen)
        if case["way"] == "step":
            state["leaves"] = [state[k].requires_grad_() for k in ("x", "residual") if state[k] is not None]
        return state
    batch, queries, keys, dim = (case[k] for k in ("batch", "queries", "keys", "dim"))
    heads, kv_heads = case["heads"], case["kv_heads"]
    # scores as a trained layer has them: a few keys stand out for each query
    if case["fused"]:
        both = normal(batch, queries, heads + 2 * kv_heads, dim).mul_(1.2).to(dtype)
        q, k, v = both.split([heads, kv_heads, kv_heads], 2)
    else:
        q = (1.2 * normal(batch, queries, heads, dim)).to(dtype)
        k = (1.2 * normal(batch, keys, kv_heads, dim)).to(dtype)
        v = normal(batch, keys, kv_heads, dim).to(dtype)
    state.update(q=q, k=k, v=v, mask=make_mask(case, gen), scale=dim ** -0.5)
    if case["way"] != "forward":
        state["grad"] = (0.05 * normal(batch, queries, heads * dim)).to(dtype)
    if case["way"] == "backward":  # what the forward pass left
        out, lse = definition(state, case)
        state["out"], state["lse"] = out.to(dtype), lse.float()
    if case["way"] == "step":
        state["leaves"] = [state[n].detach().requires_grad_() for n in ("q", "k", "v")]
    return state


def run(state):
    if own:
        return run_own(state)
    with torch.no_grad():
        return plain_attend(state) if state["case"]["op"] == "attend" else plain_drop(state)


def run_own(state):
    from scale_deformable_attention_msda_gb300 import binding
    case = state["case"]
    if case["op"] == "drop":
        out = binding.dropout(state["x"], case["p"], state["counter"], residual=state["residual"])
        if case["way"] == "forward":
            return [out]
        return [out.detach()] + list(torch.autograd.grad(out, state["leaves"], state["grad"]))
    if case["way"] == "backward":
        return list(binding.msda_attention_backward(state["grad"], state["q"], state["k"], state["v"], state["out"], state["lse"],
                                                    mask=state["mask"], scale=state["scale"]))
    if case["way"] == "forward":
        return [binding.attention(state["q"], state["k"], state["v"], mask=state["mask"], scale=state["scale"])]
    out = binding.attention(*state["leaves"], mask=state["mask"], scale=state["scale"])
    return [out.detach()] + list(torch.autograd.grad(out, state["leaves"], state["grad"]))


def plain_attend(state):
    case, dtype = state["case"], state["q"].dtype
    shared = case["heads"] // case["kv_heads"]
    q = state["q"].float().transpose(1, 2)                                    # (batch, heads, queries, dim)
    k = state["k"].float().transpose(1, 2).repeat_interleave(shared, 1)
    v = state["v"].float().transpose(1, 2).repeat_interleave(shared, 1)
    batch, heads, queries, dim = q.shape
    keys = k.shape[2]
    s = torch.matmul(q, k.transpose(2, 3)) * state["scale"]
    if state["mask"] is not None:
        s = torch.where(state["mask"], s, -math.inf)
    if case["way"] == "backward":
        p = torch.where(s == -math.inf, 0.0, torch.exp(s - state["lse"][..., None]))
        out = state["out"].float().view(batch, queries, heads, dim).transpose(1, 2)
        outs = []
    else:
        top = s.amax(-1, keepdim=True)
        e = torch.exp(s - torch.where(top == -math.inf, 0.0, top))
        total = e.sum(-1, keepdim=True)
        p = e / torch.where(total == 0, 1.0, total)                           # a row that attends nothing is zero
        out = torch.matmul(p, v)
        outs = [out.transpose(1, 2).reshape(batch, queries, heads * dim).to(dtype)]
    if case["way"] == "forward":
        return outs
    g = state["grad"].float().view(batch, queries, heads, dim).transpose(1, 2)
    dv = torch.matmul(p.transpose(2, 3), g)
    ds = p * (torch.matmul(g, v.transpose(2, 3)) - (g * out).sum(-1, keepdim=True)) * state["scale"]
    dq = torch.matmul(ds, k)
    dk = torch.matmul(ds.transpose(2, 3), q)
    dk, dv = (t.view(batch, case["kv_heads"], shared, keys, dim).sum(2) for t in (dk, dv))
    return outs + [t.transpose(1, 2).contiguous().to(dtype) for t in (dq, dk, dv)]


MASK32 = 0xFFFFFFFF


def plain_keep(state, count):
    """Which of `count` entries stay: Philox4x32-10 of (entry / 8, draw number) under the seed,
    two entries of 16 bits to each of its four words."""
    threshold = round(state["case"]["p"] * 65536)
    seed, number = state["counter"][0], state["counter"][1]
    block = torch.arange((count + 7) // 8, device="cuda")
    words = [block & MASK32, block >> 32, (number & MASK32).expand_as(block), ((number >> 32) & MASK32).expand_as(block)]
    low, high = seed & MASK32, (seed >> 32) & MASK32
    for turn in range(10):
        first, second = words[0] * 0xD2511F53, words[2] * 0xCD9E8D57
        words = [((second >> 32) & MASK32) ^ words[1] ^ ((low + turn * 0x9E3779B9) & MASK32), second & MASK32,
                 ((first >> 32) & MASK32) ^ words[3] ^ ((high + turn * 0xBB67AE85) & MASK32), first & MASK32]
    halves = [part for word in words for part in (word & 0xFFFF, word >> 16)]
    return (torch.stack(halves, 1).reshape(-1)[:count] >= threshold), (65536 / (65536 - threshold) if threshold < 65536 else 0.0)


def plain_drop(state):
    x, residual = state["x"], state["residual"]
    keep, scale = plain_keep(state, x.numel())
    keep = keep.view(x.shape)
    out = torch.where(keep, x.float() * scale, 0.0)
    if residual is not None:
        out = out + residual.float()
    outs = [out.to(x.dtype)]
    if state["case"]["way"] == "forward":
        return outs
    outs.append(torch.where(keep, state["grad"].float() * scale, 0.0).to(x.dtype))
    return outs + ([state["grad"]] if residual is not None else [])


def share_of(case):
    """The share of all pairs of query and key that the mask leaves (on average where it is drawn)."""
    if case["mask"] == "groups":
        n = case["queries"]
        front, size = denoising_groups(n)
        full, rest = divmod(front, size)
        return (n * (n - front) + full * size * size + rest * rest) / (n * n)
    # an interval of mean length share, cut at the map's borders; one in sixteen is empty
    return {"none": 1.0, "padding": case["share"], "regions": case["share"] * (1 - case["share"] / 3) * 15 / 16}[case["mask"]]


def work(case):
    e = DTYPES[case["dtype"]].itemsize
    if case["op"] == "drop":
        n = case["rows"] * case["cols"]
        step = case["way"] == "step"
        return dict(bytes=n * e * (2 + case["residual"] + 2 * step), flops=n * (2 + step))
    pairs = case["batch"] * case["heads"] * case["queries"] * case["keys"] * share_of(case)
    nq = case["batch"] * case["queries"] * case["heads"] * case["dim"]
    nk = case["batch"] * case["keys"] * case["kv_heads"] * case["dim"]
    # forward: q, k, v in, out out; backward: those, the gradient and out in, three gradients out
    tensors = {"forward": 2 * nq + 2 * nk, "backward": 4 * nq + 4 * nk, "step": 4 * nq + 4 * nk}[case["way"]]
    mask = {"none": 0, "padding": case["batch"] * case["keys"], "groups": case["queries"] * case["keys"],
            "regions": case["batch"] * case["queries"] * case["keys"]}[case["mask"]]
    stats = 4 * case["batch"] * case["heads"] * case["queries"] if case["way"] == "backward" else 0
    products = {"forward": 2, "backward": 5, "step": 7}[case["way"]]
    return dict(bytes=tensors * e + mask + stats, flops=int(2 * products * pairs * case["dim"]))


def definition(state, case, grads=False):
    """softmax(scale q k' where the mask allows) v in 64 bits, (out, log of the sums) or, with
    `grads`, (out, gradients of q, k, v) by differentiating it; one batch entry and key head at a time."""
    shared = case["heads"] // case["kv_heads"]
    parts = {n: state[n].detach().double() for n in ("q", "k", "v")}
    batch, queries, heads, dim = parts["q"].shape
    keys = parts["k"].shape[1]
    mask = state["mask"]
    mask = None if mask is None else mask.expand(batch, heads, queries, keys)
    out = torch.zeros_like(parts["q"])
    lse = torch.zeros(batch, heads, queries, device="cuda", dtype=torch.float64)
    found = {n: torch.zeros_like(parts[n]) for n in parts}
    g = state["grad"].double().view(batch, queries, heads, dim) if grads else None
    for b in range(batch):
        for n in range(case["kv_heads"]):
            mine = slice(n * shared, (n + 1) * shared)
            leaf = [parts["q"][b, :, mine].transpose(0, 1), parts["k"][b, :, n], parts["v"][b, :, n]]
            leaf = [t.clone().requires_grad_(grads) for t in leaf]
            s = state["scale"] * (leaf[0] @ leaf[1].mT)
            some = torch.ones(shared, queries, 1, dtype=torch.bool, device="cuda")
            if mask is not None:
                some = mask[b, mine].any(-1, keepdim=True)
                s = s.masked_fill(~mask[b, mine] & some, -math.inf)
            o = torch.softmax(s, -1) @ leaf[2] * some
            out[b, :, mine] = o.detach().transpose(0, 1)
            lse[b, mine] = torch.where(some, torch.logsumexp(s.detach(), -1, keepdim=True), -math.inf)[..., 0]
            if grads:
                dq, dk, dv = torch.autograd.grad(o, leaf, g[b, :, mine].transpose(0, 1))
                found["q"][b, :, mine], found["k"][b, :, n], found["v"][b, :, n] = dq.transpose(0, 1), dk, dv
    out = out.view(batch, queries, heads * dim)
    return (out, found["q"], found["k"], found["v"]) if grads else (out, lse)


def exact(case, seed):
    """The definitions in 64 bits; the generator's words on the host."""
    state = prepare(case, seed)
    if case["op"] == "attend":
        if case["way"] == "forward":
            return [definition(state, case)[0]]
        outs = list(definition(state, case, grads=True))
        return outs[1:] if case["way"] == "backward" else outs
    x = state["x"].detach()
    seed_word, number = (int(t) % 2 ** 64 for t in state["counter"].tolist())
    blocks = numpy.arange(-(-x.numel() // 8), dtype=numpy.uint64)
    half, low = numpy.uint64(32), numpy.uint64(MASK32)
    c = [blocks & low, blocks >> half, numpy.full_like(blocks, number & MASK32), numpy.full_like(blocks, number >> 32)]
    key = [seed_word & MASK32, seed_word >> 32]
    for _ in range(10):
        a, b = c[0] * numpy.uint64(0xD2511F53), c[2] * numpy.uint64(0xCD9E8D57)
        c = [(b >> half) ^ c[1] ^ numpy.uint64(key[0]), b & low, (a >> half) ^ c[3] ^ numpy.uint64(key[1]), a & low]
        key = [(key[0] + 0x9E3779B9) & MASK32, (key[1] + 0xBB67AE85) & MASK32]
    words = numpy.stack(c, 1).astype("<u4").reshape(-1).view("<u2")[: x.numel()]
    dropped = round(case["p"] * 65536)
    factor = torch.from_numpy((words >= dropped).astype(numpy.float64)).to(x.device).view(x.shape) * (65536 / max(1, 65536 - dropped))
    outs = [x.double() * factor + (0 if state["residual"] is None else state["residual"].detach().double())]
    if case["way"] == "step":
        outs += [state["grad"].double() * factor] + ([state["grad"].double()] if case["residual"] else [])
    return outs
