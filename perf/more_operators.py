"""What a training step of an MoE transformer takes beside whole-matrix Muon, AdamW and the gradient norm.

  blocks   a Muon step on weights whose blocks (the heads of an attention projection, by rows or by columns; the factors
           of an adapter) are orthogonalised one by one by Newton-Schulz products: momentum, update and weights
  balance  the balance loss of MoE routers over packed sequences, the tokens each expert got, and the gradient of the
           logits
  bias     the step of the routers' selection biases, against the sign of each expert's excess

`own` False computes the operators with elementary torch operations, `own` True calls the library.
"""

import math

import torch

own = False

LR, MOMENTUM, DECAY, GAMMA = 0.02, 0.95, 0.1, 0.2
SCHEDULE = [(3.4445, -4.7750, 2.0315)] * 8 + [(2.0, -1.5, 0.5)] * 2
COEF = 1e-3   # of the balance loss
RATE = 1e-3   # of the bias step
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # the two factors of rank-16 adapters on 27 layers' hidden states: the smallest call, fp32 weights
        _blocks("blocks: 27 adapters of rank 16", 27, 1, 16, 2048, False, param="f32", grad="f32"),
        # one query projection of the 16B-MoE model, 16 heads by rows
        _blocks("blocks: 16 heads by rows", 1, 16, 128, 2048, False),
        # one output projection, whose heads are columns
        _blocks("blocks: 16 heads by columns", 1, 16, 128, 2048, True),
        # odd sizes in rows longer than the weight, fp32 gradients, clipped, each update scaled by its own RMS
        _blocks("blocks: ragged", 3, 7, 80, 1407, True, grad="f32", pitch=13, clip=True, unit_rms=True),
        # the attention of the dense block: 4 projections of 32 heads
        _blocks("blocks: dense attention", 4, 32, 128, 4096, False),
        # every attention matrix of the 16B-MoE model
        _blocks("blocks: 27 layers of attention", 108, 16, 128, 2048, False),
        # a short microbatch through one router, fp32 logits: launches count
        _balance("balance: 512 tokens", 1, 512, 64, 6, 1, "f32", "softmax"),
        # one layer's microbatch of 16384 tokens, packed in five sequences
        _balance("balance: one layer, packed", 1, 16384, 64, 6, 5, "bf16", "softmax"),
        # all 27 layers at once, normalised sigmoid scores
        _balance("balance: 27 layers", 27, 8192, 64, 6, 4, "f32", "sigmoid"),
        # many experts, long batch with padding between the sequences' ends, odd number of sequences
        _balance("balance: 256 experts", 1, 131072, 256, 8, 37, "bf16", "sigmoid", mask=True),
        # after the step: the biases of 27 routers, and of a few large ones
        {"name": "bias: 27 routers", "op": "bias", "routers": 27, "experts": 64},
        {"name": "bias: 58 routers of 256", "op": "bias", "routers": 58, "experts": 256},
    ]


def _blocks(name, tensors, blocks, small, large, columns, param="bf16", grad="bf16", pitch=0, clip=False, unit_rms=False,
            nesterov=True):
    """`tensors` weights, each of `blocks` blocks of small x large (by rows), or large x small (by columns); rows lie
    `pitch` elements further apart than they are long."""
    return {"name": name, "op": "blocks", "tensors": tensors, "blocks": blocks, "small": small, "large": large,
            "columns": columns, "param": param, "grad": grad, "pitch": pitch, "clip": clip, "unit_rms": unit_rms,
            "nesterov": nesterov}


def _balance(name, routers, tokens, experts, top, sequences, dtype, score, mask=False):
    return {"name": name, "op": "balance", "routers": routers, "tokens": tokens, "experts": experts, "top": top,
            "sequences": sequences, "dtype": dtype, "score": score, "mask": mask}


def draw(rng):
    spread = lambda lo, hi: int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))  # noqa: E731
    op = rng.choice(("blocks", "blocks", "balance", "balance", "bias"))
    if op == "bias":
        return {"op": op, "routers": spread(1, 64), "experts": spread(2, 512)}
    if op == "balance":
        experts = spread(2, 512)
        tokens = spread(1, min(131072, (1 << 25) // experts))
        routers = max(1, min(spread(1, 32), (1 << 25) // (experts * tokens)))
        return {"op": op, "routers": routers, "tokens": tokens, "experts": experts,
                "top": min(experts, rng.randint(1, 10)), "sequences": spread(1, min(64, tokens)),
                "dtype": rng.choice(("f32", "bf16")), "score": rng.choice(("softmax", "sigmoid")),
                "mask": rng.random() < 0.3}
    small = rng.choice((16, 32, 64, 96, 128, spread(1, 128)))
    large = max(small, spread(64, 8192))
    total = spread(4e4, 1.2e8)
    blocks = max(1, min(spread(1, 40), total // (small * large)))
    tensors = max(1, min(spread(1, 60), total // (small * large * blocks)))
    case = _blocks(None, tensors, blocks, small, large, rng.random() < 0.5, rng.choice(("bf16", "bf16", "f32")),
                   rng.choice(("f32", "bf16")), rng.choice((0, 0, 8, rng.randint(1, 99))), rng.random() < 0.3,
                   rng.random() < 0.2, rng.random() < 0.8)
    del case["name"]
    return case


# ------------------------------------------------------------------------------------------------------- inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"case": case}
    make = {"blocks": _prepare_blocks, "balance": _prepare_balance, "bias": _prepare_bias}[case["op"]]
    make(s, case, gen)
    if own:
        _describe(s)
    return s


def _weight_shape(case):
    """Rows, columns and row pitch of one weight."""
    if case["columns"]:
        rows, cols = case["large"], case["blocks"] * case["small"]
    else:
        rows, cols = case["blocks"] * case["small"], case["large"]
    return rows, cols, cols + case["pitch"]


def _as_blocks(x, case):
    """The blocks of all weights (tensors x rows x cols) as one tensor of small x large matrices."""
    t, b, n, m = case["tensors"], case["blocks"], case["small"], case["large"]
    if case["columns"]:
        return x.view(t, m, b, n).permute(0, 2, 3, 1).reshape(t * b, n, m)
    return x.reshape(t * b, n, m)


def _as_weights(x, case):
    """_as_blocks' blocks back as weights."""
    t, b, n, m = case["tensors"], case["blocks"], case["small"], case["large"]
    if case["columns"]:
        return x.view(t, b, n, m).permute(0, 3, 1, 2).reshape(t, m, b * n)
    return x.view(t, b * n, m)


def _spectral(case, gen):
    """Gradients as training has them: singular values of each block spread over three decades, and noise."""
    b, n, m = case["blocks"], case["small"], case["large"]
    left = torch.randn(b, n, n, generator=gen, device="cuda") / math.sqrt(n)
    sigma = torch.exp(torch.rand(b, 1, n, generator=gen, device="cuda") * math.log(1e3) + math.log(1e-4))
    right = torch.randn(b, n, m, generator=gen, device="cuda") / math.sqrt(m)
    return torch.matmul(left * sigma, right) + torch.randn(b, n, m, generator=gen, device="cuda") * 1e-5


def _prepare_blocks(s, case, gen):
    rows, cols, pitch = _weight_shape(case)
    for kind, dtype in (("param", TYPES[case["param"]]), ("grad", TYPES[case["grad"]]), ("momentum", torch.float32)):
        s[kind] = torch.empty(case["tensors"], rows, pitch, dtype=dtype, device="cuda")
    for t in range(case["tensors"]):
        s["param"][t] = torch.randn(rows, pitch, generator=gen, device="cuda") * 0.02
        for kind, scale in (("grad", 1.0), ("momentum", 4.0)):  # a momentum holds some gradients' sum
            s[kind][t] = torch.randn(rows, pitch, generator=gen, device="cuda")  # what lies behind the rows is not read
            x = _spectral(case, gen) * scale
            x = x.permute(2, 0, 1).reshape(rows, cols) if case["columns"] else x.view(rows, cols)
            s[kind][t, :, :cols] = x
    s["factor"] = torch.rand(1, generator=gen, device="cuda") * 0.9 + 0.05 if case["clip"] else None


def _prepare_balance(s, case, gen):
    routers, tokens, experts = case["routers"], case["tokens"], case["experts"]
    bias = torch.randn(routers, 1, experts, generator=gen, device="cuda") * 0.5  # experts differ in how often they win
    logits = torch.randn(routers, tokens, experts, generator=gen, device="cuda") + bias
    s["logits"] = logits.to(TYPES[case["dtype"]])
    s["chosen"] = torch.topk(s["logits"].float(), case["top"], dim=2).indices
    # sequences of all lengths; one that is empty, where there are many
    cuts = torch.rand(case["sequences"] - 1, generator=gen, device="cuda").mul(tokens + 1).long().sort().values
    ends = torch.tensor([tokens], device="cuda")
    s["offsets"] = torch.cat([ends * 0, cuts, ends]).int()
    if case["sequences"] > 8:
        s["offsets"][4] = s["offsets"][5]
    # the last eighth of each 64 tokens is padding in a padded batch
    s["mask"] = torch.arange(tokens, device="cuda") % 64 < 56 if case["mask"] else None
    s["counts"] = torch.zeros(routers, experts, dtype=torch.int64, device="cuda")
    s["loss"] = torch.zeros(routers, device="cuda")
    s["dlogits"] = torch.zeros_like(s["logits"])


def _prepare_bias(s, case, gen):
    shape = (case["routers"], case["experts"])
    s["bias"] = torch.randn(shape, generator=gen, device="cuda") * 0.01
    mean = 4096.0 * torch.exp(torch.randn(shape, generator=gen, device="cuda") * 0.3)
    s["counts"] = mean.long()
    s["counts"][:, ::7] = 4096  # loads that may meet the mean


def _describe(s):
    """The context and the descriptors that a program makes once and keeps."""
    import muon_step_amd as ms

    case = s["case"]
    s["ctx"] = ms.Context(0)
    if case["op"] == "blocks":
        cols = _weight_shape(case)[1]
        shape = (case["large"], case["small"]) if case["columns"] else (case["small"], case["large"])
        s["table"] = ms.table(
            ms.block_matrix(s["param"][t, :, :cols], s["grad"][t, :, :cols], s["momentum"][t, :, :cols], *shape)
            for t in range(case["tensors"]))
        s["hp"] = ms.make_hparams(
            lr=LR, momentum=MOMENTUM, weight_decay=DECAY, gamma=GAMMA, nesterov=case["nesterov"], coeffs=SCHEDULE,
            scale_mode=ms.MUON_SCALE_UNIT_RMS if case["unit_rms"] else ms.MUON_SCALE_SQRT_MAX, grad_factor=s["factor"])
    elif case["op"] == "balance":
        s["table"] = ms.table(
            ms.router(s["logits"][r], s["chosen"][r], s["counts"][r], s["loss"][r:r + 1], dlogits=s["dlogits"][r],
                      offsets=s["offsets"], mask=s["mask"]) for r in range(case["routers"]))
        s["hp"] = ms.balance_hparams(
            coef=COEF, score=ms.MUON_SCORE_SIGMOID if case["score"] == "sigmoid" else ms.MUON_SCORE_SOFTMAX)
    else:
        s["table"] = ms.table(ms.router_bias(s["bias"][r], s["counts"][r]) for r in range(case["routers"]))


# ---------------------------------------------------------------------------------------------------- one pass

def run(s):
    op = s["case"]["op"]
    if op == "blocks":
        s["ctx"].muon_blocks_step(s["table"], s["hp"]) if own else _plain_blocks(s)
        return {"param": s["param"], "momentum": s["momentum"]}
    if op == "balance":
        s["ctx"].muon_router_balance(s["table"], s["hp"]) if own else _plain_balance(s)
        return {"loss": s["loss"], "counts": s["counts"], "dlogits": s["dlogits"]}
    if own:
        s["ctx"].muon_router_bias_step(s["table"], RATE)
    else:
        excess = s["counts"].shape[1] * s["counts"] - s["counts"].sum(1, keepdim=True)
        s["bias"] -= RATE * torch.sign(excess).float()
    return s["bias"]


def _plain_blocks(s):
    case = s["case"]
    cols = _weight_shape(case)[1]
    w, momentum = s["param"][:, :, :cols], s["momentum"][:, :, :cols]
    g = s["grad"][:, :, :cols].float()
    if s["factor"] is not None:
        g = g * s["factor"]
    momentum.mul_(MOMENTUM).add_(g)
    x = _as_blocks((MOMENTUM * momentum + g) if case["nesterov"] else momentum.contiguous(), case)
    x = x / x.square().sum((1, 2), keepdim=True).sqrt()
    for a, b, c in SCHEDULE:
        gram = torch.matmul(x, x.transpose(1, 2).contiguous())
        x = a * x + torch.matmul(b * gram + c * torch.matmul(gram, gram), x)
    if case["unit_rms"]:
        scale = GAMMA / x.square().mean((1, 2), keepdim=True).sqrt()
    else:
        scale = GAMMA * math.sqrt(max(case["small"], case["large"]))
    w.copy_((1 - LR * DECAY) * w.float() - LR * _as_weights(x * scale, case))


def _sequence_of(s):
    """The sequence of each token (the last that begins at or before it and is not empty)."""
    at = torch.arange(s["case"]["tokens"], device="cuda")
    return (at[:, None] >= s["offsets"][None, 1:]).sum(1)


def _plain_balance(s):
    case = s["case"]
    routers, tokens, experts, top, sequences = (case[k] for k in ("routers", "tokens", "experts", "top", "sequences"))
    sequence = _sequence_of(s)
    taking = torch.ones(tokens, device="cuda") if s["mask"] is None else s["mask"].float()
    length = torch.zeros(sequences, device="cuda").index_add_(0, sequence, taking)
    weight = COEF / (length > 0).sum()
    row = torch.arange(routers, device="cuda")[:, None] * sequences + sequence  # of counts: router and sequence
    counts = torch.zeros(routers * sequences * experts, device="cuda")
    places = row[:, :, None] * experts + s["chosen"]
    counts.index_add_(0, places.flatten(), taking[:, None].expand(routers, tokens, top).flatten())
    counts = counts.view(routers, sequences, experts)
    s["counts"].copy_(counts.sum(1))
    x = s["logits"].float()
    score = torch.log(torch.sigmoid(x)) if case["score"] == "sigmoid" else x
    p = torch.exp(score - score.max(2, keepdim=True).values)
    p = p / p.sum(2, keepdim=True)
    # the loss is the sum over tokens of the sum over experts of factor p; a row's probabilities sum to 1, so its
    # gradient takes the factors without their mean, which would only cancel
    mean = counts.mean(2, keepdim=True)
    unit = (weight * experts / top / length.square().clamp(min=1))[:, None]
    away = (unit * (counts - mean))[:, sequence]
    dot = (away * p).sum(2, keepdim=True)
    s["loss"].copy_(((dot + (unit * mean)[:, sequence]) * taking[:, None]).double().sum((1, 2)))
    d = p * (away - dot) * taking[:, None]
    s["dlogits"].copy_(d * torch.sigmoid(-x) if case["score"] == "sigmoid" else d)


# ------------------------------------------------------------------------------------------ what it takes, exactly

def work(case):
    if case["op"] == "bias":
        return {"bytes": 16 * case["routers"] * case["experts"], "flops": 4 * case["routers"] * case["experts"]}
    if case["op"] == "balance":
        rows = case["routers"] * case["tokens"]
        extra = case["tokens"] if case["mask"] else 0
        small = case["routers"] * (8 * case["experts"] + 4) + 4 * (case["sequences"] + 1)
        return {"bytes": rows * (2 * TYPES[case["dtype"]].itemsize * case["experts"] + 8 * case["top"]) + small + extra,
                "flops": 12 * rows * case["experts"]}
    n, m = case["small"], case["large"]
    blocks = case["tensors"] * case["blocks"]
    each = 8 + TYPES[case["grad"]].itemsize + 2 * TYPES[case["param"]].itemsize
    # one triangle of the first product, polynomials of small x small matrices (three products a step, one triangle
    # each), and one product with the update
    flops = n * (n + 1) * m + len(SCHEDULE) * 3 * n * n * (n + 1) + 2 * n * n * m
    return {"bytes": blocks * n * m * each, "flops": blocks * flops}


def exact(case, seed):
    s = prepare(case, seed)
    return {"blocks": _exact_blocks, "balance": _exact_balance, "bias": _exact_bias}[case["op"]](s, case)


def _exact_bias(s, case):
    counts = s["counts"].double()
    step = (counts < counts.mean(1, keepdim=True)).double() - (counts > counts.mean(1, keepdim=True)).double()
    return s["bias"].double() + RATE * step


def _exact_blocks(s, case):
    """Block by block, from the side of the larger number of rows: X (a + b G + c G^2) with G the smaller Gram matrix."""
    cols = _weight_shape(case)[1]
    param, momentum = s["param"].double(), s["momentum"].double()
    factor = 1.0 if s["factor"] is None else s["factor"].double()
    n, m = case["small"], case["large"]
    for t in range(case["tensors"]):
        g = s["grad"][t, :, :cols].double()
        if s["factor"] is not None:
            g = (g * factor).float().double()  # the clipped gradient is an fp32 value
        new = MOMENTUM * momentum[t, :, :cols] + g
        momentum[t, :, :cols] = new
        inputs = MOMENTUM * new + g if case["nesterov"] else new
        for first in range(0, case["blocks"] * n, n):
            tall = inputs[:, first:first + n] if case["columns"] else inputs[first:first + n].T
            y = tall / torch.linalg.matrix_norm(tall)
            for a, b, c in SCHEDULE:
                gram = y.T @ y
                poly = c * gram @ gram + b * gram
                poly.diagonal().add_(a)
                y = y @ poly
            rms = torch.linalg.matrix_norm(y) / math.sqrt(n * m)
            y = y * (LR * GAMMA * (1 / rms if case["unit_rms"] else math.sqrt(max(n, m))))
            place = param[t, :, first:first + n] if case["columns"] else param[t, first:first + n, :cols].T
            place.mul_(1 - LR * DECAY).sub_(y)
    return {"param": param, "momentum": momentum}


def _exact_balance(s, case):
    experts, top = case["experts"], case["top"]
    tokens = [] if s["mask"] is None else s["mask"].cpu()
    starts = s["offsets"].tolist()
    kept = []  # the tokens of each sequence that has any
    for lo, hi in zip(starts, starts[1:]):
        at = torch.arange(lo, hi)
        at = at[tokens[lo:hi]] if s["mask"] is not None else at
        if len(at):
            kept.append(at.cuda())
    loss = torch.zeros(case["routers"], dtype=torch.float64, device="cuda")
    counts = torch.zeros_like(s["counts"])
    dlogits = torch.zeros(s["logits"].shape, dtype=torch.float64, device="cuda")
    for r in range(case["routers"]):
        for at in kept:
            x = s["logits"][r, at].double()
            if case["score"] == "sigmoid":
                score = 1 / (1 + torch.exp(-x))
                p = score / score.sum(1, keepdim=True)
            else:
                p = torch.softmax(x, 1)
            got = torch.bincount(s["chosen"][r, at].flatten(), minlength=experts)
            counts[r] += got
            load = got.double() * experts / (top * len(at))
            loss[r] += COEF / len(kept) * (load * p.mean(0)).sum()
            c = COEF / len(kept) / len(at) * load
            grad = p * (c - (p * c).sum(1, keepdim=True))
            dlogits[r, at] = grad / (1 + torch.exp(x)) if case["score"] == "sigmoid" else grad
    return {"loss": loss, "counts": counts, "dlogits": dlogits}
