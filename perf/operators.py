"""Training the feed-forward of a DiT block: the gated feed-forward block, its backward pass and the AdamW step.

A case is one call sequence of a user's program:

    ffn      y = (silu(x Wg^T) * (x Wu^T)) Wd^T, with the pre-activation u = [x Wg^T | x Wu^T] kept for the backward
             pass (training) or not (serving)
    ffn_bwd  dx, dW_up, dW_down from dy, x, u and the weights
    adamw    one optimizer step over many tensors: (optionally) the global gradient norm and its clip factor, then AdamW
             on f32 parameters, with an optional bf16 copy of each and with the two moments in f32 or in 8 bits

Sizes are those of this repository: d 5120, width 13,824 (256 and 512 in the tiny workload), 31,248 tokens of the
low-resolution grid, 1,252 audio tokens of a packed sample, 4,099 tokens and d 1000 of the ragged tests.

The moments in 8 bits.  A tensor is cut into blocks of 256 values, each with one f32 scale s, the block's largest
magnitude.  A first moment is stored as a sign and k in 0..127 and stands for sign * (k/127)^2 * s, a second moment as
k in 0..255 and stands for (k/255)^4 * s.  A value between two neighbours lo and hi becomes hi where
r * (hi - lo) < value - lo, with r a 16-bit fraction, so that its expectation is the value; a positive second moment is
stored as 1 at least, so that it never divides by nothing.  The fractions come from a 32-bit hash of the seed, the step,
the tensor's number and the element's index in it (the two halves of the hash: first moment, second moment).
"""
import math
import random

import torch

own = False

BETA1, BETA2, EPS, LR, STEP, DECAY, MAX_NORM, SEED = 0.9, 0.999, 1e-8, 1e-4, 10, 0.01, 1.0, 20240229
BLOCK = 256


def listed():
    return [
        # one token through the block's feed-forward (a denoising server's smallest batch): the weights' bytes count
        {"name": "ffn_token", "op": "ffn", "tokens": 1, "d": 5120, "inner": 13824, "keep": False, "pad": 0},
        # the tiny workload, for training: launch latency counts
        {"name": "ffn_tiny", "op": "ffn", "tokens": 32, "d": 256, "inner": 512, "keep": True, "pad": 0},
        # the audio tokens of one packed sample, for training
        {"name": "ffn_audio", "op": "ffn", "tokens": 1252, "d": 5120, "inner": 13824, "keep": True, "pad": 0},
        # the low-resolution grid, for training
        {"name": "ffn_lowres", "op": "ffn", "tokens": 31248, "d": 5120, "inner": 13824, "keep": True, "pad": 0},
        # the same three for the backward pass
        {"name": "ffn_bwd_tiny", "op": "ffn_bwd", "tokens": 32, "d": 256, "inner": 512, "pad": 0},
        {"name": "ffn_bwd_audio", "op": "ffn_bwd", "tokens": 1252, "d": 5120, "inner": 13824, "pad": 0},
        {"name": "ffn_bwd_lowres", "op": "ffn_bwd", "tokens": 31248, "d": 5120, "inner": 13824, "pad": 0},
        # ragged in every direction: rows that are slices of wider ones, widths that end inside a tile
        {"name": "ffn_bwd_ragged", "op": "ffn_bwd", "tokens": 4099, "d": 1000, "inner": 2504, "pad": 8},
        # the small parameters of many blocks (norm weights, biases, adapters): many tensors, little in each
        {"name": "adamw_many", "op": "adamw", "count": 160, "low": 100, "high": 20000, "pattern": 1, "bits": 32,
         "grad": "f32", "copy": False, "clip": True},
        # both weights of one feed-forward, with the bf16 copy that the linear layers read
        {"name": "adamw_ffn", "op": "adamw", "d": 5120, "inner": 13824, "bits": 32, "grad": "bf16", "copy": True,
         "clip": True},
        # the moments in 8 bits: some odd-sized tensors, and both weights of one feed-forward
        {"name": "adamw8_some", "op": "adamw", "count": 12, "low": 1000, "high": 400000, "pattern": 2, "bits": 8,
         "grad": "f32", "copy": False, "clip": False},
        {"name": "adamw8_ffn", "op": "adamw", "d": 5120, "inner": 13824, "bits": 8, "grad": "bf16", "copy": True,
         "clip": True},
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(("ffn", "ffn_bwd", "adamw"))
    if op != "adamw":
        case = {"op": op, "tokens": spread(1, 8192), "d": 8 * spread(8, 640), "inner": 8 * spread(8, 1728),
                "pad": rng.choice((0, 0, 8, 24))}
        if op == "ffn":
            case["keep"] = rng.random() < 0.6
        return case
    low = spread(1, 100000)
    return {"op": op, "count": spread(1, 200), "low": low, "high": low * spread(1, 30) + 1, "pattern": rng.randrange(1 << 20),
            "bits": rng.choice((8, 32)), "grad": rng.choice(("f32", "bf16")), "copy": rng.random() < 0.5,
            "clip": rng.random() < 0.5}


def sizes_of(case):
    if "d" in case:
        return [2 * case["inner"] * case["d"], case["d"] * case["inner"]]
    r = random.Random(case["pattern"])
    return [max(1, int(math.exp(r.uniform(math.log(case["low"]), math.log(case["high"]))))) for _ in range(case["count"])]


def work(case):
    if case["op"] == "adamw":
        n = sum(sizes_of(case))
        grad = 2 if case["grad"] == "bf16" else 4
        # p read and written, the gradient, the moments read and written, the copy; moments in 8 bits are also given as
        # the bf16 values they stand for
        per = 8 + grad + (16 if case["bits"] == 32 else 4 + 4) + (2 if case["copy"] else 0)
        return {"bytes": per * n, "flops": 16 * n}
    t, d, inner = case["tokens"], case["d"], case["inner"]
    if case["op"] == "ffn":
        return {"bytes": 2 * (2 * t * d + 3 * inner * d + (2 * t * inner if case["keep"] else 0)), "flops": 6 * t * d * inner}
    return {"bytes": 2 * (3 * t * d + 2 * t * inner + 6 * inner * d), "flops": 12 * t * d * inner}


def drawn(g, rows, cols, pad, std):
    """A bf16 [rows, cols] tensor, a slice of rows that are `pad` wider."""
    t = torch.empty((rows, cols + pad), device="cuda", dtype=torch.bfloat16)
    return t.normal_(0.0, std, generator=g)[:, :cols]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    state = {"case": case}
    if case["op"] == "adamw":
        return prepare_adamw(case, g, state)
    t, d, inner, pad = case["tokens"], case["d"], case["inner"], case["pad"]
    state["x"] = drawn(g, t, d, pad, 1.0)
    state["w_up"] = drawn(g, 2 * inner, d, pad, d ** -0.5)
    state["w_down"] = drawn(g, d, inner, pad, inner ** -0.5)
    if case["op"] == "ffn":
        state["y"] = torch.empty((t, d), device="cuda", dtype=torch.bfloat16)
        state["u"] = torch.empty((t, 2 * inner), device="cuda", dtype=torch.bfloat16) if case["keep"] else None
    else:
        state["dy"] = drawn(g, t, d, pad, 0.01)
        state["u"] = drawn(g, t, 2 * inner, pad, 1.0)
        state["dx"] = torch.empty((t, d), device="cuda", dtype=torch.bfloat16)
        state["dw_up"] = torch.empty((2 * inner, d), device="cuda", dtype=torch.bfloat16)
        state["dw_down"] = torch.empty((d, inner), device="cuda", dtype=torch.bfloat16)
    if own:
        from dit_block_b200 import train
        state["workspace"] = train.ffn_workspace(t, d, inner)
    return state


def prepare_adamw(case, g, state):
    # the tensors of a kind lie in one allocation, each from a multiple of 256 values on; what is between them is zero
    sizes = sizes_of(case)
    starts, total = [], 0
    for n in sizes:
        starts.append(total)
        total += -(-n // BLOCK) * BLOCK
    one = lambda dtype=torch.float32: torch.zeros(total, device="cuda", dtype=dtype)  # noqa: E731
    used = one(torch.bool)
    index = torch.arange(total, device="cuda", dtype=torch.int64)
    which = one(torch.int32)
    decay = one()
    for j, (s, n) in enumerate(zip(starts, sizes)):
        used[s:s + n] = True
        index[s:s + -(-n // BLOCK) * BLOCK] -= s
        which[s:s + -(-n // BLOCK) * BLOCK] = j
        decay[s:s + n] = DECAY if n > 5120 else 0.0  # small parameters are not decayed
    normal = lambda std: one().normal_(0.0, std, generator=g).mul_(used)  # noqa: E731
    state["p"] = normal(0.02)
    # gradients whose scale differs from block to block, as those of rows of a weight do
    scale = torch.exp(torch.randn(total // BLOCK, 1, device="cuda", generator=g)).mul_(1e-4)
    grad = (normal(1.0).view(-1, BLOCK) * scale).view(-1)
    state["grad"] = grad.bfloat16() if case["grad"] == "bf16" else grad
    # moments as a run of such gradients leaves them
    m = (normal(0.23).view(-1, BLOCK) * scale).view(-1)
    v = ((0.01 * (1 + 0.3 * normal(1.0).abs()) * used).view(-1, BLOCK) * scale * scale).view(-1)
    del grad, scale
    state["copy"] = one(torch.bfloat16) if case["copy"] else None
    if case["bits"] == 32:
        state["m"], state["v"], state["m_scale"], state["v_scale"] = m, v, None, None
        del index, which
    else:
        r = torch.full_like(m, 0.5)
        state["m"], state["m_scale"] = encode_first(m, r)
        state["v"], state["v_scale"] = encode_second(v, r)
        state["m_value"], state["v_value"] = one(torch.bfloat16), one(torch.bfloat16)
        state["index"], state["which"] = index.to(torch.int32), which
    state["decay"], state["norm"] = decay, torch.zeros(2, device="cuda")
    if own:
        from dit_block_b200 import train
        cut = lambda t: None if t is None else [t[s:s + n] for s, n in zip(starts, sizes)]  # noqa: E731
        cut_scales = lambda t: None if t is None else [t[s // BLOCK:s // BLOCK + -(-n // BLOCK)] for s, n in zip(starts, sizes)]  # noqa: E731
        state["optimizer"] = train.AdamW(cut(state["p"]), cut(state["grad"]), cut(state["m"]), cut(state["v"]),
                                         m_scales=cut_scales(state["m_scale"]), v_scales=cut_scales(state["v_scale"]),
                                         copies=cut(state["copy"]),
                                         weight_decay=[DECAY if n > 5120 else 0.0 for n in sizes])
        state["workspace"] = state["optimizer"].norm_workspace()
    return state


def run(state):
    if own:
        return run_own(state)
    case = state["case"]
    if case["op"] == "ffn":
        return plain_ffn(state)
    if case["op"] == "ffn_bwd":
        return plain_ffn_bwd(state)
    return plain_adamw(state)


def run_own(state):
    from dit_block_b200 import train
    case = state["case"]
    if case["op"] == "ffn":
        train.ffn(state["y"], state["x"], state["w_up"], state["w_down"], u=state["u"], workspace=state["workspace"])
        return {"y": state["y"], "u": state["u"]}
    if case["op"] == "ffn_bwd":
        train.ffn_backward(state["dy"], state["x"], state["u"], state["w_up"], state["w_down"], dx=state["dx"],
                           dw_up=state["dw_up"], dw_down=state["dw_down"], workspace=state["workspace"])
        return {"dx": state["dx"], "dw_up": state["dw_up"], "dw_down": state["dw_down"]}
    optimizer = state["optimizer"]
    if case["clip"]:
        optimizer.grad_norm(state["norm"], MAX_NORM, workspace=state["workspace"])
    optimizer.step(lr=LR, betas=(BETA1, BETA2), eps=EPS, step=STEP, seed=SEED,
                   grad_factor=state["norm"][1:] if case["clip"] else None)
    m, v = state["m"], state["v"]
    if case["bits"] == 8:
        m, v = state["m_value"], state["v_value"]
        train.adamw_state_decode(m, v, state["m"], state["v"], state["m_scale"], state["v_scale"])
    return {"p": state["p"], "copy": state["copy"], "m": m, "v": v, "norm": state["norm"] if case["clip"] else None}


# The plain forms.

def plain_ffn(state):
    x, w_up, w_down = state["x"].float(), state["w_up"].float(), state["w_down"].float()
    u = x @ w_up.t()
    inner = w_down.shape[1]
    a, b = u[:, :inner], u[:, inner:]
    y = (a / (1 + torch.exp(-a)) * b) @ w_down.t()
    state["y"].copy_(y)
    if state["u"] is not None:
        state["u"].copy_(u)
    return {"y": state["y"], "u": state["u"]}


def plain_ffn_bwd(state):
    dy, x, u = state["dy"].float(), state["x"].float(), state["u"].float()
    w_up, w_down = state["w_up"].float(), state["w_down"].float()
    inner = w_down.shape[1]
    a, b = u[:, :inner], u[:, inner:]
    s = 1 / (1 + torch.exp(-a))
    d_act = dy @ w_down
    state["dw_down"].copy_(dy.t() @ (a * s * b))
    du = torch.cat([d_act * b * s * (1 + a * (1 - s)), d_act * a * s], dim=1)
    state["dx"].copy_(du @ w_up)
    state["dw_up"].copy_(du.t() @ x)
    return {"dx": state["dx"], "dw_up": state["dw_up"], "dw_down": state["dw_down"]}


def mixed(h):
    """A 32-bit integer mixed (the finalizer of MurmurHash3, Appleby 2011), on integers of 64 bits."""
    h = ((h ^ (h >> 16)) * 0x85EBCA6B) & 0xFFFFFFFF
    h = ((h ^ (h >> 13)) * 0xC2B2AE35) & 0xFFFFFFFF
    return h ^ (h >> 16)


def fractions(index, which):
    """The two 16-bit fractions of each element: of the first and of the second moment."""
    key = mixed((which.long() * 0x9E3779B9 + STEP) & 0xFFFFFFFF)
    key = mixed(mixed(key ^ (SEED >> 32)) ^ (SEED & 0xFFFFFFFF))
    h = mixed((index.long() + mixed(key)) & 0xFFFFFFFF)
    return (h >> 16).float() / 65536, (h & 0xFFFF).float() / 65536


def encode_first(m, r):
    blocks = m.view(-1, BLOCK)
    s = blocks.abs().amax(dim=1, keepdim=True)
    t = (blocks.abs() / torch.where(s > 0, s, 1)) * 16129
    k = torch.floor(torch.sqrt(t))
    k = torch.where(r.view(-1, BLOCK) * (2 * k + 1) < t - k * k, k + 1, k).clamp(max=127)
    return (k * torch.sign(blocks)).to(torch.int8).view(-1), s.view(-1)


def encode_second(v, r):
    blocks = v.view(-1, BLOCK)
    s = blocks.amax(dim=1, keepdim=True)
    t = (blocks / torch.where(s > 0, s, 1)) * 4228250625.0
    k = torch.floor(torch.sqrt(torch.sqrt(t)))
    width = ((4 * k + 6) * k + 4) * k + 1
    k = torch.where(r.view(-1, BLOCK) * width < t - (k * k) * (k * k), k + 1, k).clamp(max=255)
    k = torch.where(blocks > 0, k.clamp(min=1), k)
    return k.to(torch.uint8).view(-1), s.view(-1)


def decode_first(q, s):
    k = q.float().view(-1, BLOCK) / 127
    return (k * k.abs() * s[:, None]).view(-1)


def decode_second(q, s):
    k = q.float().view(-1, BLOCK) / 255
    return ((k * k) * (k * k) * s[:, None]).view(-1)


def plain_adamw(state):
    case = state["case"]
    grad = state["grad"].float()
    if case["clip"]:
        norm = torch.sqrt(grad.double().square().sum())
        state["norm"].copy_(torch.stack([norm, torch.clamp(MAX_NORM / (norm + 1e-6), max=1.0)]))
        grad = grad * state["norm"][1]
    m, v = state["m"], state["v"]
    if case["bits"] == 8:
        m, v = decode_first(m, state["m_scale"]), decode_second(v, state["v_scale"])
    m = m * BETA1 + grad * (1 - BETA1)
    v = v * BETA2 + grad * grad * (1 - BETA2)
    p = state["p"]
    p.sub_(LR * (state["decay"] * p + m / (1 - BETA1 ** STEP) / (torch.sqrt(v / (1 - BETA2 ** STEP)) + EPS)))
    if case["copy"]:
        state["copy"].copy_(p)
    if case["bits"] == 8:
        rm, rv = fractions(state["index"], state["which"])
        q, s = encode_first(m, rm)
        state["m"].copy_(q), state["m_scale"].copy_(s)
        q, s = encode_second(v, rv)
        state["v"].copy_(q), state["v_scale"].copy_(s)
        # 7 and 8 bits a value: bf16 tells every two of the values that a block can hold apart
        state["m_value"].copy_(decode_first(state["m"], state["m_scale"]))
        state["v_value"].copy_(decode_second(state["v"], state["v_scale"]))
        m, v = state["m_value"], state["v_value"]
    else:
        state["m"].copy_(m), state["v"].copy_(v)
        m, v = state["m"], state["v"]
    return {"p": p, "copy": state["copy"], "m": m, "v": v, "norm": state["norm"] if case["clip"] else None}


# The definitions, in 64 bits.

def exact(case, seed):
    s = prepare(case, seed)
    f = lambda name: s[name].to(torch.float64)  # noqa: E731
    if case["op"] == "adamw":
        return exact_adamw(case, s, f)
    inner = case["inner"]
    if case["op"] == "ffn":
        u = torch.matmul(f("x"), f("w_up").T)
        gate, up = u.split(inner, dim=1)
        return {"y": torch.matmul(gate * torch.sigmoid(gate) * up, f("w_down").T), "u": u if case["keep"] else None}
    gate, up = f("u").split(inner, dim=1)
    sig = torch.sigmoid(gate)
    out = {"dw_down": torch.matmul(f("dy").T, gate * sig * up)}
    down = torch.matmul(f("dy"), f("w_down"))
    # d silu(z) / dz = sig(z) + z sig(z) sig(-z)
    du = torch.empty_like(s["u"], dtype=torch.float64)
    du[:, :inner] = down * up * (sig + gate * sig * torch.sigmoid(-gate))
    du[:, inner:] = down * gate * sig
    del down, sig, gate, up
    out["dx"] = torch.matmul(du, f("w_up"))
    out["dw_up"] = torch.matmul(du.T, f("x"))
    return out


def exact_adamw(case, s, f):
    p, g = f("p"), f("grad")
    norm = None
    if case["clip"]:
        length = torch.linalg.vector_norm(g)
        norm = torch.stack([length, (MAX_NORM / (length + 1e-6)).clamp(max=1.0)])
        g = g * norm[1]
    if case["bits"] == 32:
        m, v = f("m"), f("v")
    else:
        q = f("m").reshape(-1, BLOCK)
        m = (torch.sign(q) * (q / 127) ** 2 * f("m_scale").unsqueeze(1)).flatten()
        v = ((f("v").reshape(-1, BLOCK) / 255) ** 4 * f("v_scale").unsqueeze(1)).flatten()
    m = torch.lerp(g, m, BETA1)
    v = torch.lerp(g ** 2, v, BETA2)
    denominator = torch.sqrt(v / (1 - BETA2 ** STEP)) + EPS
    p = p - LR * f("decay") * p - LR * m / (1 - BETA1 ** STEP) / denominator
    if case["bits"] == 8:
        r1, r2 = fractions(s["index"], s["which"])
        m = torch.sign(m) * rounded(m.abs(), r1.double(), 127, 2)
        v = rounded(v, r2.double(), 255, 4, least=1)
    return {"p": p, "copy": p if case["copy"] else None, "m": m, "v": v, "norm": norm}


def rounded(x, r, top, power, least=0):
    """x >= 0 in blocks of 256, each value one of (k / top)^power * max, rounded up where the fraction r says so."""
    x = x.reshape(-1, BLOCK)
    s = x.max(dim=1, keepdim=True).values
    unit = x / torch.where(s == 0, torch.ones_like(s), s)
    grid = (torch.arange(top + 2, device=x.device, dtype=torch.float64) / top) ** power
    low = torch.searchsorted(grid, unit, right=True) - 1
    up = r.reshape(-1, BLOCK) * (grid[low + 1] - grid[low]) < unit - grid[low]
    k = (low + up).clamp(max=top)
    if least:
        k = torch.where(x > 0, k.clamp(min=least), k)
    return (grid[k] * s).flatten()
