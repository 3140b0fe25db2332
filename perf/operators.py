"""The operators of an optimizer step on the tensors that take AdamW, and the gradient clip in front of every step.

  norm     the 2-norm of all gradients together, and the factor that clips it to `max_norm`
  adamw32  one AdamW step over many tensors, moments in 32 bits; bf16 or fp32 weights and gradients, optionally with
           fp32 master weights beside bf16 ones
  adamw8   the same step with both moments in 8 bits: e4m3 codes with one power-of-two scale (an e8m0 byte) for each 32
           elements of a tensor, rounded stochastically

The tensors of a case are views of one flat buffer for each kind of data, each starting at a multiple of 64 elements, as a
program with flattened parameters keeps them; what lies between them is left as it was.  `own` False computes the
operators with elementary torch operations, `own` True calls the library.
"""

import math

import torch

own = False

LR, BETA1, BETA2, EPS, DECAY = 0.02, 0.9, 0.95, 1e-8, 0.1
MAX_NORM = 1.0
SEED = 20240917  # of the stochastic rounding: the same number a training run would keep
BLOCK = 32       # elements of one 8-bit block
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    vocabulary, hidden, expert = 102400, 2048, 2048 * 1408
    return [
        # the norm weights of 27 layers and the last one: small tensors, where the call's latency counts
        _norm("norm: 55 norm weights", f"55*{hidden}", "f32"),
        # every matrix of one 16B-MoE layer: 4 of attention, 64 experts of 3
        _norm("norm: one MoE layer", f"4*{hidden * hidden}+192*{expert}", "bf16"),
        # the dense block's matrices
        _norm("norm: dense block", f"4*{4096 * 4096}+3*{4096 * 14336}", "bf16"),
        # embedding and head, gradients accumulated in fp32
        _norm("norm: embedding and head", f"2*{vocabulary * hidden}", "f32"),
        _adamw("adamw32: 55 norm weights", "adamw32", f"55*{hidden}", "bf16", True, "bf16", True, 1),
        # the routers of 27 layers (64 experts), fp32 weights and bf16 gradients
        _adamw("adamw32: routers", "adamw32", f"27*{64 * hidden}", "f32", False, "bf16", True, 1000),
        # odd sizes, bf16 weights without a master copy, fp32 gradients
        _adamw("adamw32: ragged", "adamw32", "9*1+11*1407+5*10001+2*4194301", "bf16", False, "f32", False, 7),
        # the embedding in mixed precision: bf16 weights, fp32 master weights, bf16 gradients
        _adamw("adamw32: embedding", "adamw32", f"1*{vocabulary * hidden}", "bf16", True, "bf16", True, 1000),
        _adamw("adamw8: 55 norm weights", "adamw8", f"55*{hidden}", "bf16", True, "bf16", True, 1),
        _adamw("adamw8: ragged", "adamw8", "9*1+11*1407+5*10001+2*4194301", "f32", False, "f32", False, 7),
        # the embedding with the fewest bytes: bf16 weights and gradients, 8-bit moments
        _adamw("adamw8: embedding", "adamw8", f"1*{vocabulary * hidden}", "bf16", False, "bf16", True, 1000),
        # the head with fp32 master weights and gradients accumulated in fp32
        _adamw("adamw8: head, master", "adamw8", f"1*{vocabulary * hidden}", "bf16", True, "f32", True, 1000),
    ]


def _norm(name, sizes, grad):
    return {"name": name, "op": "norm", "sizes": sizes, "grad": grad}


def _adamw(name, op, sizes, param, master, grad, clip, step):
    return {"name": name, "op": op, "sizes": sizes, "param": param, "master": master, "grad": grad, "clip": clip,
            "step": step}


def draw(rng):
    op = rng.choice(("norm", "adamw32", "adamw8"))
    kinds = rng.randint(1, 3)
    total = math.exp(rng.uniform(math.log(2e3), math.log(1.2e8)))
    sizes = []
    for _ in range(kinds):
        count = max(1, int(math.exp(rng.uniform(0, math.log(60)))))
        each = max(1, int(total / kinds / count * rng.uniform(0.5, 1.0)))
        sizes.append(f"{count}*{each + rng.choice((0, 1, -each % 2048))}")
    case = {"op": op, "sizes": "+".join(sizes), "grad": rng.choice(("f32", "bf16"))}
    if op != "norm":
        param = rng.choice(("f32", "bf16"))
        case.update(param=param, master=param == "bf16" and rng.random() < 0.5, clip=rng.random() < 0.5,
                    step=rng.choice((1, 2, 30, 1000, 200000)))
    return case


# ------------------------------------------------------------------------------------------------------- inputs

def _numels(case):
    parts = [p.split("*") for p in case["sizes"].split("+")]
    return [int(n) for c, n in parts for _ in range(int(c))]


def _starts(numels):
    at, total = [], 0
    for n in numels:
        at.append(total)
        total += -(-n // 64) * 64
    return at, total


def _noise(numels, starts, total, gen):
    """Standard normal values whose rows of 2048 have scales of their own (a quarter of the rows of a large buffer is
    zero: the rows of tokens that a batch does not hold), zero between the tensors."""
    x = torch.randn(total, generator=gen, device="cuda")
    rows = -(-total // 2048)
    scale = torch.exp(torch.randn(rows, generator=gen, device="cuda"))
    if rows > 1000:
        scale *= (torch.rand(rows, generator=gen, device="cuda") > 0.25).float()
    x *= scale.repeat_interleave(2048)[:total]
    for n, at in zip(numels, starts):
        x[at + n:at + (-(-n // 64) * 64)] = 0
    return x


def _block_exponents(largest):
    """The e8m0 byte of blocks whose largest magnitude is `largest` (fp32): 2^(e-127) brings it to (224, 448]."""
    return (((largest.view(torch.int32) + 0x1FFFFF) >> 23) - 8).clamp(min=17)


def _eight_bits(x, floor):
    """fp32 values as a checkpoint in 8 bits holds them: (codes, exponents), rounded to nearest."""
    x = x.reshape(-1, BLOCK)
    largest = x.abs().amax(1)
    e = _block_exponents(largest)
    y = x * ((254 - e) << 23).view(torch.float32)[:, None]
    if floor:
        y = torch.where((largest > 0)[:, None], y.clamp(min=2.0 ** -9), y)
    return y.to(torch.float8_e4m3fn).reshape(-1), e.to(torch.uint8)


def _element(s):
    """The place of each element of the flat buffers in its own tensor, and which of them belong to one."""
    i = torch.empty(s["grad"].numel(), dtype=torch.int64, device="cuda")
    inside = torch.zeros(s["grad"].numel(), dtype=torch.bool, device="cuda")
    for n, at in zip(s["numels"], s["starts"]):
        room = -(-n // 64) * 64
        torch.arange(room, out=i[at:at + room])
        inside[at:at + n] = True
    return i, inside


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    numels = _numels(case)
    starts, total = _starts(numels)
    grad = (_noise(numels, starts, total, gen) * 1e-3).to(TYPES[case["grad"]])
    s = {"case": case, "numels": numels, "starts": starts, "grad": grad}
    if case["op"] == "norm":
        s["norm"] = torch.zeros(1, dtype=torch.float64, device="cuda")
        s["factor"] = torch.zeros(1, device="cuda")
    else:
        w = torch.randn(total, generator=gen, device="cuda") * 0.02
        s["param"] = w.to(TYPES[case["param"]])
        s["master"] = w if case["master"] else None
        s["factor"] = torch.rand(1, generator=gen, device="cuda") * 0.9 + 0.05 if case["clip"] else None
        m = _noise(numels, starts, total, gen) * 3e-4
        v = (_noise(numels, starts, total, gen) * 1e-3) ** 2 + m * m
        if case["step"] == 1:
            m.zero_()
            v.zero_()
        if case["op"] == "adamw32":
            s["exp_avg"], s["exp_avg_sq"] = m, v
        else:
            s["exp_avg"], s["exp_avg_scale"] = _eight_bits(m, False)
            s["exp_avg_sq"], s["exp_avg_sq_scale"] = _eight_bits(v, True)
            _clear_between(s, total)
    if own:
        _describe(s)
    elif case["op"] == "adamw8":
        s["element"] = _element(s)  # goes by the sizes alone: kept, as the descriptors are
    return s


def _clear_between(s, total):
    """The bytes between the tensors, which the floor of exp_avg_sq's codes may have touched, back to zero."""
    codes = s["exp_avg_sq"].view(torch.uint8)
    for n, at in zip(s["numels"], s["starts"]):
        codes[at + n:at + (-(-n // 64) * 64)] = 0


def _describe(s):
    """The context and the descriptors that a program makes once and keeps.  The weights between the tensors of a
    flattened buffer decay with the others: what lies behind a tensor is handed over as one without a gradient."""
    import muon_step_amd as ms

    case = s["case"]
    s["ctx"] = ms.Context(0)
    view = lambda name, at, n: None if s[name] is None else s[name][at:at + n]  # noqa: E731
    items = []
    for n, at in zip(s["numels"], s["starts"]):
        if case["op"] == "norm":
            items.append(ms.grad(view("grad", at, n)))
            continue
        for first, count in ((at, n), (at + n, -n % 64)):
            if count == 0:
                continue
            param, grad, master = (view(name, first, count) for name in ("param", "grad", "master"))
            m, v = view("exp_avg", first, count), view("exp_avg_sq", first, count)
            if case["op"] == "adamw32":
                items.append(ms.adamw_mixed_tensor(param, grad, m, v, master=master))
                continue
            if first == at:
                blocks = -(-n // BLOCK)
                m_scale, v_scale = (view(name + "_scale", at // BLOCK, blocks) for name in ("exp_avg", "exp_avg_sq"))
            else:  # moments of zero, whose exponents nothing else reads
                m_scale, v_scale = (torch.zeros(2, dtype=torch.uint8, device="cuda")[:-(-count // BLOCK)] for _ in range(2))
            items.append(ms.adamw8_tensor(param, grad, (m, m_scale, v, v_scale), master=master))
    s["table"] = ms.table(items)
    if case["op"] != "norm":
        s["hp"] = ms.adamw_hparams(lr=LR, beta1=BETA1, beta2=BETA2, eps=EPS, weight_decay=DECAY, step=case["step"])


# ---------------------------------------------------------------------------------------------------- one pass

def run(s):
    op = s["case"]["op"]
    if op == "norm":
        if own:
            s["ctx"].muon_grad_norm(s["table"], MAX_NORM, s["norm"], s["factor"])
        else:
            norm = s["grad"].double().square().sum().sqrt().reshape(1)
            s["norm"] = norm
            s["factor"] = torch.where(norm > MAX_NORM, MAX_NORM / norm, torch.ones_like(norm)).float()
        return {"norm": s["norm"], "factor": s["factor"]}
    if own:
        if op == "adamw32":
            s["ctx"].muon_adamw_mixed_step(s["table"], s["hp"], grad_factor=s["factor"])
        else:
            s["ctx"].muon_adamw8_step(s["table"], s["hp"], seed=SEED, grad_factor=s["factor"])
    elif op == "adamw32":
        m, v = _moments(s, s["exp_avg"], s["exp_avg_sq"])
        _update(s, m, v)
        s["exp_avg"].copy_(m)
        s["exp_avg_sq"].copy_(v)
    else:
        _plain8(s)
    out = {k: s[k] for k in ("param", "master", "exp_avg", "exp_avg_sq")}
    if op == "adamw8":
        out["exp_avg_scale"] = s["exp_avg_scale"].view(torch.float8_e8m0fnu)
        out["exp_avg_sq_scale"] = s["exp_avg_sq_scale"].view(torch.float8_e8m0fnu)
    return out


def _moments(s, m, v):
    g = s["grad"].float()
    if s["factor"] is not None:
        g = g * s["factor"]
    return BETA1 * m + (1 - BETA1) * g, BETA2 * v + ((1 - BETA2) * g) * g


def _update(s, m, v):
    step = s["case"]["step"]
    w = s["master"] if s["master"] is not None else s["param"].float()
    denominator = (v / (1 - BETA2 ** step)).sqrt() + EPS
    w = (1 - LR * DECAY) * w - LR * ((m / (1 - BETA1 ** step)) / denominator)
    if s["master"] is not None:
        s["master"].copy_(w)
    s["param"].copy_(w)


def _mix(x):
    """32-bit mixing of int64 values below 2^32."""
    x = x ^ (x >> 16)
    x = (x * 0x6A09E667) & 0xFFFFFFFF
    x = x ^ (x >> 15)
    x = (x * 0xBB67AE85) & 0xFFFFFFFF
    return x ^ (x >> 16)


def _key(seed, step):
    return _mix((seed & 0xFFFFFFFF) ^ _mix((seed >> 32) ^ _mix((step & 0xFFFFFFFF) ^ _mix(step >> 32))))


def _stochastic(x, e, turn, i, hashed, floor):
    """x 2^(127-e) to e4m3: away from zero where the part that is cut off, in steps of the code, and a random number
    below 1 (20 bits of the group's hash, turned by 8 for each element and by `turn`) sum to 1 or more."""
    turn = (8 * (i & 3) + turn) & 31
    random = (((hashed << turn) | (hashed >> (32 - turn))) & 0xFFFFFFFF) >> 12
    y = x.double().reshape(-1, BLOCK) * _power(127 - e)[:, None]
    if floor:
        y = torch.where((x.reshape(-1, BLOCK).amax(1) > 0)[:, None], y.clamp(min=2.0 ** -9), y)
    y = y.reshape(-1)
    spacing = _power((torch.frexp(y)[1] - 1).clamp(min=-6) - 3)
    code = torch.floor(y.abs() / spacing + random.double() * 2.0 ** -20) * spacing
    return torch.copysign(code, y).float().to(torch.float8_e4m3fn)


def _power(k):
    """2^k for whole numbers, exactly."""
    return ((k.long() + 1023) << 52).view(torch.float64)


def _plain8(s):
    e_m, e_v = s["exp_avg_scale"].int(), s["exp_avg_sq_scale"].int()
    old = lambda codes, e: (codes.float().reshape(-1, BLOCK) * _power(e - 127).float()[:, None]).reshape(-1)  # noqa: E731
    m, v = _moments(s, old(s["exp_avg"], e_m), old(s["exp_avg_sq"], e_v))
    _update(s, m, v)
    i, inside = s["element"]
    group = i >> 2
    key = _key(SEED, s["case"]["step"])
    hashed = _mix(((group & 0xFFFFFFFF) ^ key) ^ (((group >> 32) * 0x9E3779B9) & 0xFFFFFFFF))
    for name, x, turn, floor in (("exp_avg", m, 0, False), ("exp_avg_sq", v, 16, True)):
        e = _block_exponents(x.abs().reshape(-1, BLOCK).amax(1))
        codes = _stochastic(x, e, turn, i, hashed, floor).view(torch.uint8)
        kept = s[name].view(torch.uint8)
        kept.copy_(torch.where(inside, codes, kept))
        touched = inside.reshape(-1, BLOCK)[:, 0]
        s[name + "_scale"].copy_(torch.where(touched, e.to(torch.uint8), s[name + "_scale"]))


# ------------------------------------------------------------------------------------------ what it takes, exactly

def work(case):
    n = sum(_numels(case))
    grad = TYPES[case["grad"]].itemsize
    if case["op"] == "norm":
        return {"bytes": n * grad + 12, "flops": 2 * n}
    weights = 8 + 2 if case["master"] else 2 * TYPES[case["param"]].itemsize  # with a master the bf16 copy is only written
    moments = 16 if case["op"] == "adamw32" else 4 + 4 / BLOCK
    return {"bytes": n * (grad + weights + moments), "flops": 16 * n}


def exact(case, seed):
    s = prepare({k: case[k] for k in case}, seed)
    g = s["grad"].to(torch.float64)
    if case["op"] == "norm":
        norm = torch.linalg.vector_norm(g).cpu()
        return {"norm": norm.reshape(1), "factor": torch.clamp(MAX_NORM / norm, max=1.0).reshape(1)}
    if s["factor"] is not None:
        g = (g * s["factor"].to(torch.float64)).float().double()  # the clipped gradient is an fp32 value
    if case["op"] == "adamw32":
        m0, v0 = s["exp_avg"].double(), s["exp_avg_sq"].double()
    else:
        m0 = torch.ldexp(s["exp_avg"].double().view(-1, BLOCK), s["exp_avg_scale"].long()[:, None] - 127).flatten()
        v0 = torch.ldexp(s["exp_avg_sq"].double().view(-1, BLOCK), s["exp_avg_sq_scale"].long()[:, None] - 127).flatten()
    t = case["step"]
    m, v = m0 + (1 - BETA1) * (g - m0), v0 + (1 - BETA2) * (g * g - v0)
    w = (s["master"] if case["master"] else s["param"]).double()
    w = w - LR * DECAY * w - LR / (1 - BETA1 ** t) * m / ((v / (1 - BETA2 ** t)) ** 0.5 + EPS)
    out = {"param": w, "master": w if case["master"] else None}
    if case["op"] == "adamw32":
        return {**out, "exp_avg": m, "exp_avg_sq": v}
    # The 8-bit moments are defined as the rounding of fp32 values whose every product and sum is rounded; a value next
    # to a border would otherwise fall on its other side.
    f = lambda x: x.float().double()  # noqa: E731
    c = [f(torch.tensor(b, dtype=torch.float64, device="cuda")) for b in (BETA1, 1 - BETA1, BETA2, 1 - BETA2)]
    m, v = f(f(c[0] * m0) + f(c[1] * g)), f(f(c[2] * v0) + f(f(c[3] * g) * g))
    values = torch.arange(127, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn).double()
    for name, x, half in (("exp_avg", m, 0), ("exp_avg_sq", v, 1)):
        blocks = x.view(-1, BLOCK)
        largest = blocks.abs().amax(1, keepdim=True)
        exponent = torch.ceil(torch.log2((largest / 448).clamp(min=2.0 ** -110))).clamp(min=-110)
        y = blocks.abs() / torch.exp2(exponent)
        if half:
            y = torch.where(largest > 0, y.clamp(min=2.0 ** -9), y)
        below = torch.bucketize(y, values, right=True) - 1
        above = (below + 1).clamp(max=126)
        share = (y - values[below]) / (values[above] - values[below]).clamp(min=2.0 ** -9)
        del blocks
        up = share.flatten() + _twenty_bits(s, half) >= 1
        code = torch.where(up, values[above].flatten(), values[below].flatten()) * x.sign()
        inside = _element(s)[1]
        out[name] = torch.where(inside, code, s[name].double())
        out[name + "_scale"] = torch.where(inside[::BLOCK], torch.exp2(exponent).flatten(),
                                           torch.exp2(s[name + "_scale"].double() - 127))
    return out


def _twenty_bits(s, half):
    """The random numbers of the rounding, as multiples of 2^-20, from the hash's definition over bytes: element j of a
    group of four takes the word whose bytes are the hash's turned by j (and by two more for the second moment)."""
    i = _element(s)[0]
    word = _mix((i // 4 % 2 ** 32) ^ _key(SEED, s["case"]["step"]) ^ (i // 2 ** 34 * 0x9E3779B9 % 2 ** 32))
    turns = (i % 4 + 2 * half) % 4
    byte = lambda k: word // 256 ** ((k - turns) % 4) % 256  # noqa: E731
    turned = byte(3) * 2 ** 24 + byte(2) * 2 ** 16 + byte(1) * 2 ** 8 + byte(0)
    return (turned // 2 ** 12).double() / 2 ** 20
