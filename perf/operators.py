"""Operators of a data-parallel training step around the gradient AllReduce, as measured cases.

A training step reduces its gradients over the ranks; these are the operators
on both sides of that reduction:

- ``layer_norm``, ``layer_norm_backward``: the layer whose weight gradient is a
  sum over every token of every rank: over a rank's tokens in the backward
  pass, over the ranks in the AllReduce;
- ``grad_norm``: the global 2-norm of the reduced gradients;
- ``adamw``: the AdamW step over many tensors at once, states in float32;
- ``adamw_packed``: the same step with each state in 8 bits.

The optimizer's cases write beside their inputs (in place is the same call
without ``out``), so that a pass can be taken again on the same state.  Sizes
are this repository's gradient buckets (4 x 1,024 and 8 x 2^20 elements, shards
of 8 x 2^24) and generic shapes.

The packed states.  A block is 256 consecutive elements of a tensor; it has
one scale byte e >= 1, the value 2^(e-127) (255: the whole block is NaN), the
smallest power of two whose 1.875-fold reaches the block's largest magnitude.
The first moment's code is a sign, 4 exponent bits E and 3 mantissa bits F,
times 2^(e-127): (1 + F/8) 2^(E-15), or F/8 2^-14 at E = 0; the second
moment's has 5 exponent bits and no sign: (1 + F/8) 2^(E-31), or F/8 2^-30 at
E = 0.  A new state is rounded to one of its two neighbours, up with the
probability of its place between them, from 16 of the 32 bits that a hash gives
for (seed, tensor, element); a positive second moment is never rounded to 0.
"""

import math
import random

import torch

own = False

BLOCK = 256
BETAS, EPS, DECAY, LR, STEP, MAX_NORM, SEED = (0.9, 0.999), 1e-8, 0.1, 3e-4, 1000, 1.0, 1234
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
M32 = 0xFFFFFFFF


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def listed():
    return [
        # the smallest gradient bucket: one call's latency
        {"name": "norm 4 KiB", "op": "grad_norm", "total": 1024, "tensors": 1, "align": 64, "grad": "f32"},
        # the parameters of a few layers, back to back in their buckets, before clipping
        {"name": "norm ragged bf16", "op": "grad_norm", "total": 9_700_001, "tensors": 97, "align": 1, "grad": "bf16"},
        # eight ranks' shards of a large float32 gradient
        {"name": "norm 8 shards f32", "op": "grad_norm", "total": 1 << 27, "tensors": 8, "align": 64, "grad": "f32"},
        # one layer's vectors only: a step that is all latency
        {"name": "adamw small", "op": "adamw", "total": 4099, "tensors": 6, "align": 64, "param": "f32", "grad": "f32",
         "copy": "none"},
        # mixed precision: float32 masters, bf16 gradients and weights, ragged tensors back to back
        {"name": "adamw ragged mixed", "op": "adamw", "total": 25_000_003, "tensors": 149, "align": 1, "param": "f32",
         "grad": "bf16", "copy": "bf16"},
        # eight ranks' shards of a large float32 model after a reduce-scatter
        {"name": "adamw 8 shards f32", "op": "adamw", "total": 1 << 27, "tensors": 8, "align": 64, "param": "f32",
         "grad": "f32", "copy": "none"},
        # one bucket with states in 8 bits
        {"name": "packed bucket", "op": "adamw_packed", "total": (1 << 20) + 77, "tensors": 12, "align": 256,
         "param": "f32", "grad": "f32", "copy": "none"},
        # eight ranks' shards of a large bf16 model with states in 8 bits
        {"name": "packed 8 shards bf16", "op": "adamw_packed", "total": 1 << 27, "tensors": 8, "align": 256,
         "param": "bf16", "grad": "bf16", "copy": "none"},
        # a few tokens on each of 4 ranks
        {"name": "layer norm few rows", "op": "layer_norm", "ranks": 4, "rows": 5, "cols": 1024, "pad": 0, "dtype": "bf16"},
        # a training batch: 8 ranks x 4,096 tokens of width 4,096
        {"name": "layer norm batch bf16", "op": "layer_norm", "ranks": 8, "rows": 4096, "cols": 4096, "pad": 0,
         "dtype": "bf16"},
        # odd width and row stride in float32
        {"name": "layer norm backward odd f32", "op": "layer_norm_backward", "ranks": 7, "rows": 515, "cols": 1003,
         "pad": 5, "dtype": "f32"},
        # the same training batch, backward
        {"name": "layer norm backward batch bf16", "op": "layer_norm_backward", "ranks": 8, "rows": 4096, "cols": 4096,
         "pad": 0, "dtype": "bf16"},
    ]


def _between(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("grad_norm", "adamw", "adamw_packed", "layer_norm", "layer_norm_backward"))
    if op.startswith("layer_norm"):
        ranks, cols = rng.randint(1, 8), _between(rng, 16, 16384)
        rows = _between(rng, 1, max(1, min(32768, (1 << 26) // (ranks * cols))))
        return {"op": op, "ranks": ranks, "rows": rows, "cols": cols, "pad": rng.choice((0, 0, 1, 8)),
                "dtype": rng.choice(("f32", "bf16", "f16"))}
    case = {"op": op, "total": _between(rng, 1024, 1 << 26), "tensors": _between(rng, 1, 200),
            "align": 256 if op == "adamw_packed" else rng.choice((1, 64))}
    if op == "grad_norm":
        return dict(case, grad=rng.choice(("f32", "bf16", "f16")))
    param, grad, copy = rng.choice((("f32", "f32", "none"), ("f32", "f32", "bf16"), ("f32", "bf16", "bf16"),
                                    ("f32", "f16", "f16"), ("f32", "bf16", "none"), ("bf16", "bf16", "none"),
                                    ("bf16", "f32", "none"), ("f16", "f16", "none")))
    return dict(case, param=param, grad=grad, copy=copy)


def _sizes(case):
    """The tensors' element counts: uneven (a factor of up to about 400 apart), summing to the case's total."""
    n, total = case["tensors"], case["total"]
    rng = random.Random("%d of %d" % (n, total))
    if n <= 8:
        return [(i + 1) * total // n - i * total // n for i in range(n)]
    w = [math.exp(rng.uniform(0, 6)) for _ in range(n)]
    got = [max(1, int(x / sum(w) * (total - n))) for x in w]
    got[0] += total - sum(got)
    return got


def _spans(case):
    """(start of each tensor in its flat buffer, the sizes, the buffer's length)."""
    sizes, starts, at = _sizes(case), [], 0
    for s in sizes:
        starts.append(at)
        at += -(-s // case["align"]) * case["align"]
    return starts, sizes, at


def work(case):
    if case["op"].startswith("layer_norm"):
        n, rows, cols, e = case["ranks"], case["rows"], case["cols"], BYTES[case["dtype"]]
        passes, vectors, flops = (2, 2, 8) if case["op"] == "layer_norm" else (3, 3, 16)
        return {"bytes": n * (passes * rows * cols * e + vectors * cols * e + 8 * rows), "flops": flops * n * rows * cols}
    n = case["total"]
    if case["op"] == "grad_norm":
        return {"bytes": n * BYTES[case["grad"]] + 4, "flops": 2 * n}
    per = 2 * BYTES[case["param"]] + BYTES[case["grad"]] + BYTES.get(case["copy"], 0)
    if case["op"] == "adamw":
        return {"bytes": n * (per + 16), "flops": 18 * n}
    # codes read and written, a scale byte a block of each, and both new states read out in 16 bits
    return {"bytes": n * (per + 4 + 4) + 4 * n / BLOCK, "flops": 40 * n}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    state = {"case": dict(case)}
    if case["op"].startswith("layer_norm"):
        _prepare_norm(case, state, gen)
    else:
        _prepare_tensors(case, state, gen)
    if own:
        import ring_allreduce_reduction_virtual_amd as ar

        state["ar"] = ar
        if case["op"] == "grad_norm":
            state["plan"] = ar.ar_grad_norm_init(state["grads"])
        elif case["op"] == "adamw":
            state["plan"] = ar.ar_adamw_init(state["params"], state["grads"], state["exp_avgs"], state["exp_avg_sqs"],
                                             out=state["out"], copies=state["copies"])
        elif case["op"] == "adamw_packed":
            state["plan"] = ar.ar_adamw_packed_init(state["params"], state["grads"],
                                                    [ar.PackedState(*p) for p in state["exp_avgs"]],
                                                    [ar.PackedState(*p) for p in state["exp_avg_sqs"]],
                                                    out=(state["out"][0], [ar.PackedState(*p) for p in state["out"][1]],
                                                         [ar.PackedState(*p) for p in state["out"][2]]),
                                                    copies=state["copies"])
            state["packed_out"] = tuple([ar.PackedState(*p) for p in state["out"][k]] for k in (1, 2))
    return state


def _prepare_norm(case, state, gen):
    n, rows, cols, dt = case["ranks"], case["rows"], case["cols"], DTYPES[case["dtype"]]

    def activations(scale, shift):
        wide = torch.randn(n, rows, cols + case["pad"], device="cuda", generator=gen)
        wide = wide.mul_(scale).add_(shift).to(dt)
        return [wide[r, :, :cols] for r in range(n)]

    state["x"] = activations(1.7, 0.3)
    # every rank holds its replica of the weights
    gamma = (1 + 0.1 * torch.randn(cols, device="cuda", generator=gen)).to(dt)
    beta = (0.1 * torch.randn(cols, device="cuda", generator=gen)).to(dt)
    state["gamma"], state["beta"] = ([w.clone() for _ in range(n)] for w in (gamma, beta))
    if case["op"] == "layer_norm_backward":
        state["dy"] = activations(1e-2, 0.0)
        x = torch.stack(state["x"]).float()
        mean = x.mean(-1)
        rstd = torch.rsqrt((x - mean[..., None]).square().mean(-1) + 1e-5)
        state["mean"], state["rstd"] = list(mean.unbind(0)), list(rstd.unbind(0))


def _prepare_tensors(case, state, gen):
    starts, sizes, length = _spans(case)

    def views(flat):
        return [flat[a:a + s] for a, s in zip(starts, sizes)]

    live = torch.zeros(length, device="cuda")
    for v in views(live):
        v.fill_(1.0)
    # gradients of very different size from one stretch of parameters to the next
    size = torch.exp2(torch.randint(-14, -4, (length // 64 + 1,), device="cuda", generator=gen).float())
    size = size.repeat_interleave(64)[:length]
    grad = torch.randn(length, device="cuda", generator=gen).mul_(size).mul_(live)
    state["flat_grad"] = grad.to(DTYPES[case["grad"]])
    state["grads"] = views(state["flat_grad"])
    if case["op"] == "grad_norm":
        return
    dt = DTYPES[case["param"]]
    state["flat_param"] = torch.randn(length, device="cuda", generator=gen).mul_(0.02).mul_(live).to(dt)
    m = torch.randn(length, device="cuda", generator=gen).mul_(size).mul_(0.3).mul_(live)
    v = torch.rand(length, device="cuda", generator=gen).add_(0.5).mul_(size.square()).mul_(live)
    copy = None if case["copy"] == "none" else torch.zeros(length, dtype=DTYPES[case["copy"]], device="cuda")
    state["grad_norm"] = grad.norm().reshape(1)
    state["params"] = views(state["flat_param"])
    state["flat_out"] = [torch.zeros_like(state["flat_param"])]
    state["flat_copy"], state["copies"] = copy, None if copy is None else views(copy)
    if case["op"] == "adamw":
        state["flat_m"], state["flat_v"] = m, v
        state["exp_avgs"], state["exp_avg_sqs"] = views(m), views(v)
        state["flat_out"] += [torch.zeros_like(m), torch.zeros_like(v)]
        state["out"] = tuple(views(t) for t in state["flat_out"])
        return

    def block_views(codes, scales):
        return [(codes[a:a + s], scales[a // BLOCK:a // BLOCK + -(-s // BLOCK)]) for a, s in zip(starts, sizes)]

    half = torch.full((length // BLOCK, BLOCK), 1 << 19, dtype=torch.int32, device="cuda")
    state["m"], state["v"] = _pack(m.view(-1, BLOCK), half, 4), _pack(v.view(-1, BLOCK), half, 5)
    state["exp_avgs"], state["exp_avg_sqs"] = block_views(*state["m"]), block_views(*state["v"])
    state["m_out"], state["v_out"] = (tuple(torch.zeros_like(t) for t in state[k]) for k in ("m", "v"))
    state["out"] = (views(state["flat_out"][0]), block_views(*state["m_out"]), block_views(*state["v_out"]))
    # the new states' values, every one of which bfloat16 holds exactly
    state["flat_values"] = [torch.zeros(length, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    state["m_values"], state["v_values"] = (views(t) for t in state["flat_values"])
    # which tensor each block belongs to, and its first element there
    which = torch.repeat_interleave(torch.arange(len(sizes)), torch.tensor([-(-s // BLOCK) for s in sizes]))
    first = torch.arange(length // BLOCK) * BLOCK - torch.tensor(starts)[which]
    state["which"], state["first"] = which.cuda(), first.cuda()


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def run(state):
    case = state["case"]
    return (_own if own else _plain)[case["op"]](state)


def _hyper(state):
    return dict(step=STEP, lr=LR, betas=BETAS, eps=EPS, weight_decay=DECAY, grad_norm=state["grad_norm"],
                max_norm=MAX_NORM)


def _own_grad_norm(state):
    return state["plan"].start()


def _own_adamw(state):
    state["plan"].start(**_hyper(state))
    return _step_outputs(state, state["flat_out"][1], state["flat_out"][2])


def _own_adamw_packed(state):
    state["plan"].start(seed=SEED, **_hyper(state))
    m, v = state["packed_out"]
    state["ar"].ar_unpack_states(m, "exp_avg", outs=state["m_values"])
    state["ar"].ar_unpack_states(v, "exp_avg_sq", outs=state["v_values"])
    return _step_outputs(state, *state["flat_values"])


def _own_layer_norm(state):
    y, mean, rstd = state["ar"].ar_layer_norm(state["x"], state["gamma"], state["beta"], eps=1e-5)
    return {"y": y, "mean": mean, "rstd": rstd}


def _own_layer_norm_backward(state):
    dx, dgamma, dbeta = state["ar"].ar_layer_norm_backward(state["dy"], state["x"], state["gamma"], state["mean"],
                                                           state["rstd"])
    return {"dx": dx, "dgamma": dgamma, "dbeta": dbeta}


def _step_outputs(state, m, v):
    got = {"param": state["flat_out"][0], "exp_avg": m, "exp_avg_sq": v}
    if state["flat_copy"] is not None:
        got["copy"] = state["flat_copy"]
    return got


def _plain_grad_norm(state):
    return state["flat_grad"].float().square().sum().sqrt().reshape(1)


def _updated(state, m, v):
    """The new moments and parameters in float32, each operation rounded on its own."""
    scale = torch.clamp(MAX_NORM / (state["grad_norm"] + 1e-6), max=1.0)
    g = state["flat_grad"].float() * scale
    m = m * BETAS[0] + g * (1 - BETAS[0])
    v = v * BETAS[1] + (g * g) * (1 - BETAS[1])
    denom = torch.sqrt(v) * (1 / math.sqrt(1 - BETAS[1] ** STEP)) + EPS
    p = state["flat_param"].float() * (1 - LR * DECAY) - (m / denom) * (LR / (1 - BETAS[0] ** STEP))
    return p, m, v


def _write_params(state, p):
    state["flat_out"][0].copy_(p)
    if state["flat_copy"] is not None:
        state["flat_copy"].copy_(p)


def _plain_adamw(state):
    p, m, v = _updated(state, state["flat_m"], state["flat_v"])
    _write_params(state, p)
    state["flat_out"][1].copy_(m)
    state["flat_out"][2].copy_(v)
    return _step_outputs(state, state["flat_out"][1], state["flat_out"][2])


def _scale(e):
    return torch.where(e == 255, math.nan, torch.exp2(e.clamp(min=1).float() - 127))


def _pack(x, noise, exponent_bits):
    """Codes and scale bytes of blocks of float32 values, rounded with 20 bits of noise below the code's last bit."""
    top = (x.abs().amax(-1).view(torch.int32) + 0x000FFFFF) >> 23
    e = torch.where(top >= 255, 255, top.clamp(min=1))
    low = 2.0 ** -112 if exponent_bits == 4 else 2.0 ** -96   # the code's exponent 0 becomes float32's
    bits = (x.abs() * torch.exp2(127.0 - e.float())[:, None] * low).view(torch.int32)
    codes = (bits + noise) >> 20
    if exponent_bits == 4:
        codes = codes | ((x.view(torch.int32) >> 24) & 0x80)
    else:
        codes = torch.where(x > 0, codes.clamp(min=1), codes)
    return codes.to(torch.uint8).view(-1), e.to(torch.uint8)


def _unpack(codes, scales, exponent_bits):
    codes = codes.view(-1, BLOCK).int()
    mask, up = (0x7F, 2.0 ** 112) if exponent_bits == 4 else (0xFF, 2.0 ** 96)
    x = ((codes & mask) << 20).view(torch.float32) * up
    if exponent_bits == 4:
        x = torch.where(codes >= 0x80, -x, x)
    return (x * _scale(scales)[:, None]).view(-1)


def _hash(x):
    """A 32-bit mixing of 32-bit values held in int64."""
    x = ((x ^ (x >> 16)) * 0x7FEB352D) & M32
    x = ((x ^ (x >> 15)) * 0x846CA68B) & M32
    return x ^ (x >> 16)


def _noise(state):
    """The two states' noise for every element: 16 bits of its hash each, centred in 20 bits."""
    key = _hash((SEED + 0x9E3779B9 * (state["which"] + 1)) & M32)
    i = state["first"][:, None] + torch.arange(BLOCK, device="cuda")
    r = _hash((key[:, None] + i * 0x9E3779B9) & M32)
    return ((r & 0xFFFF) * 16 + 8).int(), ((r >> 16) * 16 + 8).int()


def _plain_adamw_packed(state):
    p, m, v = _updated(state, _unpack(*state["m"], 4), _unpack(*state["v"], 5))
    _write_params(state, p)
    noise = _noise(state)
    _write_packed(state["m_out"], state["flat_values"][0], _pack(m.view(-1, BLOCK), noise[0], 4), 4)
    _write_packed(state["v_out"], state["flat_values"][1], _pack(v.view(-1, BLOCK), noise[1], 5), 5)
    return _step_outputs(state, *state["flat_values"])


def _write_packed(to, values, made, exponent_bits):
    to[0].copy_(made[0])
    to[1].copy_(made[1])
    values.copy_(_unpack(*made, exponent_bits))


def _plain_layer_norm(state):
    x = torch.stack(state["x"]).float()
    mean = x.mean(-1)
    centred = x - mean[..., None]
    rstd = 1 / torch.sqrt(centred.square().mean(-1) + 1e-5)
    y = centred * rstd[..., None] * torch.stack(state["gamma"]).float()[:, None] \
        + torch.stack(state["beta"]).float()[:, None]
    y = y.to(state["x"][0].dtype)
    return {"y": list(y.unbind(0)), "mean": list(mean.unbind(0)), "rstd": list(rstd.unbind(0))}


def _plain_layer_norm_backward(state):
    dy, x = torch.stack(state["dy"]).float(), torch.stack(state["x"]).float()
    mean, rstd = torch.stack(state["mean"])[..., None], torch.stack(state["rstd"])[..., None]
    hat = (x - mean) * rstd
    wdy = dy * torch.stack(state["gamma"]).float()[:, None]
    dx = rstd * (wdy - wdy.mean(-1, keepdim=True) - hat * (wdy * hat).mean(-1, keepdim=True))
    dgamma, dbeta = (dy * hat).sum(1), dy.sum(1)
    dt = state["x"][0].dtype
    return {"dx": list(dx.to(dt).unbind(0)), "dgamma": list(dgamma.to(dt).unbind(0)),
            "dbeta": list(dbeta.to(dt).unbind(0))}


_plain = {"grad_norm": _plain_grad_norm, "adamw": _plain_adamw, "adamw_packed": _plain_adamw_packed,
          "layer_norm": _plain_layer_norm, "layer_norm_backward": _plain_layer_norm_backward}
_own = {"grad_norm": _own_grad_norm, "adamw": _own_adamw, "adamw_packed": _own_adamw_packed,
        "layer_norm": _own_layer_norm, "layer_norm_backward": _own_layer_norm_backward}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------

def exact(case, seed):
    global own
    kept, own = own, False
    try:
        state = prepare(case, seed)
    finally:
        own = kept
    if case["op"] == "grad_norm":
        return torch.linalg.vector_norm(state["flat_grad"].double()).reshape(1)
    if case["op"].startswith("layer_norm"):
        return _exact_norm(case, state)
    return _exact_step(case, state)


def _exact_norm(case, state):
    got = {"y": [], "mean": [], "rstd": []} if case["op"] == "layer_norm" else {"dx": [], "dgamma": [], "dbeta": []}
    for r in range(case["ranks"]):
        x, w = state["x"][r].double(), state["gamma"][r].double()
        if case["op"] == "layer_norm":
            var, mean = torch.var_mean(x, dim=1, correction=0)
            rstd = (var + 1e-5) ** -0.5
            got["y"].append(torch.addcmul(state["beta"][r].double(), (x - mean[:, None]) * rstd[:, None], w))
            got["mean"].append(mean)
            got["rstd"].append(rstd)
            continue
        dy, rstd = state["dy"][r].double(), state["rstd"][r].double()[:, None]
        hat = (x - state["mean"][r].double()[:, None]) * rstd
        got["dgamma"].append(torch.einsum("rc,rc->c", dy, hat))
        got["dbeta"].append(dy.sum(0))
        part = dy * w
        along = torch.linalg.vecdot(part, hat)[:, None] / case["cols"]
        got["dx"].append((part - part.sum(1, keepdim=True) / case["cols"] - along * hat) * rstd)
    return got


def _exact_values(codes, scales, exponent_bits):
    """Code by code from a table of the 256 values."""
    table, bias = [], 15 if exponent_bits == 4 else 31
    for c in range(256):
        sign, body = (-1.0, c - 128) if exponent_bits == 4 and c >= 128 else (1.0, c)
        e, f = divmod(body, 8)
        table.append(sign * ((8 + f) * 2.0 ** (e - bias - 3) if e else f * 2.0 ** (-bias - 2)))
    values = torch.tensor(table, dtype=torch.float64, device="cuda")[codes.long()].view(-1, BLOCK)
    return (values * torch.exp2(scales.double() - 127)[:, None]).view(-1)


def _exact_round(x, up, exponent_bits):
    """x in 64 bits to the neighbour that a place `up` in [0, 1) decides."""
    bias = 15 if exponent_bits == 4 else 31
    x = x.view(-1, BLOCK)
    top = x.abs().amax(1, keepdim=True)
    scale = torch.exp2(torch.ceil(torch.log2((top / 1.875).clamp(min=2.0 ** -126))))
    scaled = x.abs() / scale
    place = torch.floor(torch.log2(scaled.clamp(min=2.0 ** (1 - bias))))
    step = torch.exp2(place - 3)
    got = torch.floor(scaled / step + up) * step
    if exponent_bits == 5:
        got = torch.where(x > 0, got.clamp(min=2.0 ** (-bias - 2)), got)
    return (torch.sign(x) * got * scale).view(-1)


def _exact_step(case, state):
    packed = case["op"] == "adamw_packed"
    g = state["flat_grad"].double() * min(1.0, MAX_NORM / (state["grad_norm"].double().item() + 1e-6))
    if packed:
        m, v = _exact_values(*state["m"], 4), _exact_values(*state["v"], 5)
    else:
        m, v = state["flat_m"].double(), state["flat_v"].double()
    m = torch.lerp(g, m, BETAS[0])
    v = torch.lerp(g.square(), v, BETAS[1])
    step = (m / (1 - BETAS[0] ** STEP)) / ((v / (1 - BETAS[1] ** STEP)).sqrt() + EPS)
    p = state["flat_param"].double()
    p = p - LR * DECAY * p - LR * step
    if packed:
        noise = _noise(state)
        m = _exact_round(m, noise[0].double() / (1 << 20), 4)
        v = _exact_round(v, noise[1].double() / (1 << 20), 5)
    got = {"param": p, "exp_avg": m, "exp_avg_sq": v}
    if case["copy"] != "none":
        got["copy"] = p
    return got
