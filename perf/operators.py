"""Operators of a linear layer trained and served in low precision, and the
loss it is tuned with: their measured cases and plain forms.

Four operators:

- ``store``: rows kept as microscaled 4-bit (MXFP4) or 8-bit (MXFP8) floats and
  read back.  Each block of 32 elements of a row has one power-of-two scale.
- ``linear``: y = Q4(x) W4^T, the product of activations quantised in the call
  with weights that are kept in MXFP4.
- ``backward``: the layer's backward pass from an 8-bit activation checkpoint:
  dx = dy W4 and dW = dy^T Q8(x).
- ``preference``: the loss of paired log ratios and its gradient in the logits.

The stored form of a rows x cols matrix: ld = cols rounded up to 128; codes
uint8 [rows, ld / 2] (MXFP4, the even element in the low nibble) or [rows, ld]
(MXFP8); scales uint8 [rows, ld / 32], the float exponent byte of each block;
zeros in the padding, whose scale byte is 1.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
BLOCK = 32
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
LARGEST = {"mx4": 6.0, "mx8": 448.0}


def listed():
    return [
        # a mini-batch of 2000-feature rows (the epsilon-shaped data set's width) kept in 4 bits: launch latency counts
        {"name": "store-mx4-small", "op": "store", "fmt": "mx4", "rows": 64, "cols": 2000, "dtype": "bf16"},
        # a layer's float32 master weights requantised after an optimiser step
        {"name": "store-mx4-weights", "op": "store", "fmt": "mx4", "rows": 8192, "cols": 8192, "dtype": "fp32"},
        # activations of a ragged batch checkpointed in 8 bits and restored
        {"name": "store-mx8-odd", "op": "store", "fmt": "mx8", "rows": 5001, "cols": 4100, "dtype": "fp16"},
        # one token through one layer: the smallest call of serving
        {"name": "linear-decode-1", "op": "linear", "m": 1, "k": 4096, "n": 4096, "dtype": "bf16", "out": "bf16"},
        # a batch of decoding sequences through a wide layer, bound by reading the weights
        {"name": "linear-decode-24", "op": "linear", "m": 24, "k": 8192, "n": 16384, "dtype": "bf16", "out": "bf16"},
        # a ragged prompt, an odd output width, float32 logits
        {"name": "linear-odd", "op": "linear", "m": 777, "k": 2000, "n": 5001, "dtype": "fp16", "out": "fp32"},
        # a full training batch through a square layer: the largest product
        {"name": "linear-large", "op": "linear", "m": 8192, "k": 8192, "n": 8192, "dtype": "bf16", "out": "bf16"},
        # a few tokens' gradients in float32 through a narrow layer
        {"name": "backward-small", "op": "backward", "m": 37, "k": 2000, "n": 1000, "dtype": "fp32", "out": "fp32"},
        # a training batch through a square layer
        {"name": "backward-large", "op": "backward", "m": 4096, "k": 4096, "n": 8192, "dtype": "bf16", "out": "bf16"},
        # two short pairs over a small vocabulary, float32 logits
        {"name": "preference-small", "op": "preference", "pairs": 2, "tokens": 61, "vocab": 2000, "stride": 2000,
         "dtype": "fp32", "loss": "logistic", "smoothing": 0.0, "average": False, "beta": 0.1},
        # an odd vocabulary inside padded rows, the squared loss of averaged ratios
        {"name": "preference-odd", "op": "preference", "pairs": 5, "tokens": 1100, "vocab": 50001, "stride": 50048,
         "dtype": "fp16", "loss": "squared", "smoothing": 0.0, "average": True, "beta": 0.5},
        # a training batch of long pairs over a large vocabulary
        {"name": "preference-large", "op": "preference", "pairs": 16, "tokens": 8192, "vocab": 65536, "stride": 65536,
         "dtype": "bf16", "loss": "logistic", "smoothing": 0.1, "average": False, "beta": 0.1},
    ]


def draw(rng):
    def size(lo, hi):  # spread over the logarithm, odd sizes included
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(["store", "linear", "linear", "backward", "preference"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op == "store":
        return {"op": op, "fmt": rng.choice(["mx4", "mx8"]), "rows": size(1, 8192), "cols": size(1, 8192), "dtype": dtype}
    if op in ("linear", "backward"):
        hi = 8192 if op == "linear" else 4096
        return {"op": op, "m": size(1, hi), "k": size(32, hi), "n": size(32, 8192), "dtype": dtype,
                "out": rng.choice([dtype, "fp32"])}
    pairs = size(1, 16)
    vocab = size(128, 65536)
    tokens = max(2 * pairs, min(size(2 * pairs, 8192), (1 << 28) // vocab))
    return {"op": op, "pairs": pairs, "tokens": tokens, "vocab": vocab, "stride": vocab + rng.choice([0, 0, 7, 64]),
            "dtype": dtype, "loss": rng.choice(["logistic", "logistic", "squared"]),
            "smoothing": rng.choice([0.0, 0.1]), "average": rng.choice([False, True]), "beta": rng.choice([0.05, 0.1, 0.5])}


def pitch(cols):
    return (cols + 127) // 128 * 128


# ---------------------------------------------------------------- inputs

def activations(shape, gen, dtype):
    """Normal values with a few channels far above the rest, as layers see them."""
    x = torch.randn(shape, generator=gen, device="cuda")
    gain = torch.where(torch.rand((1, shape[1]), generator=gen, device="cuda") < 0.02, 12.0, 1.0)
    return (x * gain).to(dtype)


def loss_scale(case):
    """fp16 gradients are taken of a scaled loss, as their range needs it."""
    return 4096.0 if case["dtype"] == "fp16" else 1.0


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype = DTYPES[case["dtype"]]
    state = {"case": case}
    if case["op"] == "store":
        state["x"] = activations((case["rows"], case["cols"]), gen, dtype)
    elif case["op"] in ("linear", "backward"):
        m, k, n = case["m"], case["k"], case["n"]
        state["x"] = activations((m, k), gen, dtype)
        weight = torch.randn((n, k), generator=gen, device="cuda") / math.sqrt(k)
        state["codes"], state["scales"] = quantize(weight, "mx4")  # laid out once, as a served layer keeps them
        if case["op"] == "backward":
            rows = torch.exp(torch.randn((m, 1), generator=gen, device="cuda"))
            state["dy"] = (torch.randn((m, n), generator=gen, device="cuda") * rows * 1e-3).to(dtype)
    else:
        t, v, pairs = case["tokens"], case["vocab"], case["pairs"]
        pad = torch.randn((t, case["stride"]), generator=gen, device="cuda") * 2.5
        state["logits"] = pad.to(dtype)[:, :v]
        # ragged sequences, each with one token at least; its first part is the prompt, which is masked
        cut = torch.randperm(t - 1, generator=gen, device="cuda")[:2 * pairs - 1].sort().values + 1
        zero = torch.zeros(1, dtype=torch.int64, device="cuda")
        state["offsets"] = torch.cat([zero, cut, zero + t])
        labels = torch.randint(0, v, (t,), generator=gen, device="cuda")
        start = state["offsets"][:-1].repeat_interleave(state["offsets"].diff())
        length = state["offsets"].diff().repeat_interleave(state["offsets"].diff())
        position = torch.arange(t, device="cuda") - start
        state["labels"] = torch.where(position * 4 < length - 1, -100, labels)
        # the reference model's log probabilities of the same tokens
        z = state["logits"].gather(1, labels[:, None])[:, 0].float()
        mean = math.log(v) + 2.5 ** 2 / 2
        noise = torch.randn(t, generator=gen, device="cuda") * 0.3
        state["ref"] = torch.where(state["labels"] < 0, 0.0, z - mean + noise)
        state["grad_loss"] = torch.full((pairs,), loss_scale(case) / pairs, device="cuda")
    return state


# ---------------------------------------------------------------- one pass

def run(state):
    case = state["case"]
    if own:
        return run_own(state, case)
    if case["op"] == "store":
        x = state["x"]
        codes, scales = quantize(x, case["fmt"])
        return dequantize(codes, scales, x.shape[1], case["fmt"]).to(x.dtype)
    if case["op"] == "linear":
        x, out = state["x"], DTYPES[case["out"]]
        x4 = dequantize(*quantize(x, "mx4"), x.shape[1], "mx4")
        w4 = dequantize(state["codes"], state["scales"], x.shape[1], "mx4")
        return (x4 @ w4.t()).to(out)
    if case["op"] == "backward":
        x, out = state["x"], DTYPES[case["out"]]
        x8 = dequantize(*quantize(x, "mx8"), x.shape[1], "mx8")
        w4 = dequantize(state["codes"], state["scales"], x.shape[1], "mx4")
        dy = state["dy"].float()
        return {"dx": (dy @ w4).to(out), "dw": dy.t() @ x8}
    return preference(state, case)


def run_own(state, case):
    from communication_avoiding_mixed_amd import binding as B

    if case["op"] == "store":
        x = state["x"]
        return B.mx_dequantize(B.mx_quantize(x, case["fmt"]), x.dtype)
    if case["op"] in ("linear", "backward"):
        w4 = B.MXMatrix("mx4", state["codes"], state["scales"], case["k"])
        out = DTYPES[case["out"]]
        if case["op"] == "linear":
            return B.mx4_linear(state["x"], w4, out)
        x8 = B.mx_quantize(state["x"], "mx8")
        return {"dx": B.mx4_grad_input(state["dy"], w4, out), "dw": B.mx8_grad_weight(state["dy"], x8)}
    fwd = B.pref_loss(state["logits"], state["labels"], state["offsets"], state["ref"], case["beta"],
                      loss=case["loss"], smoothing=case["smoothing"] if case["loss"] == "logistic" else 0.0,
                      average=case["average"])
    return {"loss": fwd.loss, "logps": fwd.logps, "dlogits": B.pref_grad(fwd, state["grad_loss"])}


# ---------------------------------------------------------------- plain forms

def power(e):
    """2^e in float32 from the exponent's bits, e in [-126, 127] (a library pow need not be exact)."""
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def quantize(x, fmt):
    """(codes, scales) of x in 32 bits.  Scale: the largest power of two with
    max|x| times it at most the largest element; elements to nearest even."""
    rows, cols = x.shape
    ld = pitch(cols)
    b = torch.zeros((rows, ld), dtype=torch.float32, device=x.device)
    b[:, :cols] = x
    b = b.view(rows, ld // BLOCK, BLOCK)
    top = b.abs().amax(2)
    mant, exp = torch.frexp(top)  # top = mant 2^exp, mant in [1/2, 1)
    if fmt == "mx4":
        e = exp - 3 + (mant > 0.75)  # 6 = 0.75 * 2^3
    else:
        e = exp - 9 + (mant > 0.875)  # 448 = 0.875 * 2^9
    e = torch.where(top > 0, e, -126).clamp(-126, 126)
    b = (b * power(-e)[:, :, None]).view(rows, ld)
    sign = torch.signbit(b).to(torch.int32)
    # |b| as a whole number of quanta 2^q, q least for subnormal values; a carry into the next binade is in the code's own order
    least, digits = (-1, 2) if fmt == "mx4" else (-9, 8)
    q = (torch.frexp(b)[1] - int(math.log2(digits)) - 1).clamp(min=least)
    code = torch.round(b.abs() * power(-q)).to(torch.int32) + (q - least) * digits
    if fmt == "mx4":
        code = (code + sign * 8).view(rows, ld // 2, 2)
        codes = (code[:, :, 0] + code[:, :, 1] * 16).to(torch.uint8)
    else:
        codes = (code + sign * 128).to(torch.uint8)
    return codes, (e + 127).to(torch.uint8)


def dequantize(codes, scales, cols, fmt):
    rows = codes.shape[0]
    if fmt == "mx4":
        both = torch.stack([codes & 15, codes >> 4], 2).view(rows, -1)
        table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float32, device=codes.device)
        value = table[both.to(torch.int32)]
    else:
        c = codes.to(torch.int32)
        e, f = (c >> 3) & 15, c & 7
        value = torch.where(e > 0, (8 + f) * power(e - 10), f * 2.0 ** -9)
        value = torch.where(c > 127, -value, value)
    scale = power(scales.to(torch.int32) - 127)
    return (value.view(rows, -1, BLOCK) * scale[:, :, None]).view(rows, -1)[:, :cols]


def preference(state, case):
    logits, labels, offsets = state["logits"], state["labels"], state["offsets"]
    keep = labels >= 0
    index = labels.clamp(min=0)[:, None]
    z = logits.float()
    top = z.amax(1, keepdim=True)
    z = z - top
    p = torch.exp(z)
    total = p.sum(1, keepdim=True)
    logps = torch.where(keep, z.gather(1, index)[:, 0] - torch.log(total)[:, 0], 0.0)
    # sums over a sequence in 64 bits, by differences of running sums
    zero = torch.zeros(1, dtype=torch.float64, device=z.device)
    ratio = torch.where(keep, logps.double() - state["ref"].double(), 0.0)
    run_sum = torch.cat([zero, ratio.cumsum(0)])[offsets].diff()
    count = torch.cat([zero, keep.double().cumsum(0)])[offsets].diff()
    per = 1.0 / count.clamp(min=1.0) if case["average"] else torch.ones_like(count)
    mean = run_sum * per
    h = mean[0::2] - mean[1::2]
    beta, eps = case["beta"], case["smoothing"]
    if case["loss"] == "logistic":
        u = beta * h
        softplus = u.abs().neg().exp().log1p()
        loss = (1 - eps) * (softplus + (-u).clamp(min=0)) + eps * (softplus + u.clamp(min=0))
        slope = beta * (eps - 1 / (1 + u.exp()))
    else:
        loss = (h - 1 / (2 * beta)) ** 2
        slope = 2 * (h - 1 / (2 * beta))
    slope = slope * state["grad_loss"].double()
    by_sequence = torch.stack([slope, -slope], 1).view(-1) * per
    coef = torch.where(keep, by_sequence.repeat_interleave(offsets.diff(), output_size=labels.shape[0]), 0.0).float()
    d = p * (-coef[:, None] / total)
    d.scatter_add_(1, index, coef[:, None])
    return {"loss": loss.float(), "logps": logps, "dlogits": d.to(logits.dtype)}


# ---------------------------------------------------------------- work

def work(case):
    if case["op"] == "store":
        count = case["rows"] * case["cols"]
        kept = 17 / 32 if case["fmt"] == "mx4" else 33 / 32
        return {"bytes": int(count * (2 * SIZE[case["dtype"]] + kept)), "flops": 0}
    if case["op"] in ("linear", "backward"):
        m, k, n = case["m"], case["k"], case["n"]
        e, eo, w = SIZE[case["dtype"]], SIZE[case["out"]], 17 / 32 * n * k
        if case["op"] == "linear":
            return {"bytes": int(e * m * k + w + eo * m * n), "flops": 2 * m * n * k}
        return {"bytes": int(e * m * (k + n) + w + eo * m * k + 4 * n * k), "flops": 4 * m * n * k}
    return {"bytes": 2 * SIZE[case["dtype"]] * case["tokens"] * case["vocab"] + 20 * case["tokens"],
            "flops": 8 * case["tokens"] * case["vocab"]}


# ---------------------------------------------------------------- 64 bits

def rounded(x, largest, bits, lowest):
    """x in blocks of 32 as its stored values: 2^e with e the least with
    max|x| <= largest 2^e, elements rounded to `bits` significant bits and no
    finer than 2^lowest of the scale."""
    x = x.double()
    rows, cols = x.shape
    blocks = torch.nn.functional.pad(x, (0, -cols % BLOCK)).reshape(rows, -1, BLOCK)
    amax = blocks.abs().max(dim=2, keepdim=True).values
    up = torch.tensor([2.0 ** e for e in range(-300, 301)], dtype=torch.float64, device=x.device)  # exact powers
    at = torch.floor(torch.log2(torch.where(amax > 0, amax, 1.0) / largest)).long() + 299
    at += (amax > largest * up[at]).long()
    at += (amax > largest * up[at]).long()
    u = blocks / up[at]
    magnitude = u.abs().clamp(min=2.0 ** -60)
    top = torch.floor(torch.log2(magnitude)).long() + 300
    top -= (up[top] > magnitude).long()
    top += (up[top + 1] <= magnitude).long()
    quantum = up[(top - (bits - 1)).clamp(min=300 + lowest)]
    return (torch.round(u / quantum) * quantum * up[at]).reshape(rows, -1)[:, :cols]


def kept_weights(state, cols):
    """The kept weights' values, from their bytes."""
    codes, scales = state["codes"].long(), state["scales"].long()
    nibbles = torch.empty((codes.shape[0], 2 * codes.shape[1]), dtype=torch.long, device=codes.device)
    nibbles[:, 0::2], nibbles[:, 1::2] = codes % 16, codes // 16
    exponent, half = nibbles % 8 // 2, (nibbles % 2).double() / 2
    size = torch.where(exponent > 0, (1 + half) * (1 << (exponent - 1).clamp(min=0)), half)
    size = torch.where(nibbles >= 8, -size, size)
    up = torch.tensor([2.0 ** (e - 127) for e in range(256)], dtype=torch.float64, device=codes.device)
    return (size * up[scales].repeat_interleave(BLOCK, dim=1))[:, :cols]


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "store":
        return rounded(state["x"], 6.0, 2, -1) if case["fmt"] == "mx4" else rounded(state["x"], 448.0, 4, -9)
    if case["op"] == "linear":
        return rounded(state["x"], 6.0, 2, -1) @ kept_weights(state, case["k"]).t()
    if case["op"] == "backward":
        dy = state["dy"].double()
        return {"dx": dy @ kept_weights(state, case["k"]), "dw": dy.t() @ rounded(state["x"], 448.0, 4, -9)}
    labels, bounds = state["labels"], state["offsets"].tolist()
    logits = state["logits"]
    t = case["tokens"]
    dlogits = torch.empty((t, case["vocab"]), dtype=torch.float64, device="cuda")
    logps = torch.zeros(t, dtype=torch.float64, device="cuda")
    losses = []
    for pair in range(case["pairs"]):
        margin, weight = 0.0, []
        for side in (0, 1):
            a, b = bounds[2 * pair + side], bounds[2 * pair + side + 1]
            logp = torch.log_softmax(logits[a:b].double(), dim=1)
            used = labels[a:b] >= 0
            rows = torch.nonzero(used)[:, 0]
            logps[a + rows] = logp[rows, labels[a + rows]]
            share = 1.0 / max(1, int(used.sum())) if case["average"] else 1.0
            margin += (1, -1)[side] * share * float((logps[a + rows] - state["ref"][a + rows].double()).sum())
            weight.append((1, -1)[side] * share)
            onehot_less = -torch.exp(logp)
            onehot_less[rows, labels[a + rows]] += 1
            onehot_less[~used] = 0
            dlogits[a:b] = onehot_less
        beta, eps = case["beta"], case["smoothing"]
        if case["loss"] == "logistic":
            plus, minus = (math.log1p(math.exp(-abs(beta * margin))) + max(0.0, s * beta * margin) for s in (1, -1))
            losses.append((1 - eps) * minus + eps * plus)
            lower = math.exp(-plus)  # the logistic function of -beta margin
            slope = beta * (eps - lower)
        else:
            losses.append((margin - 0.5 / beta) ** 2)
            slope = 2 * (margin - 0.5 / beta)
        for side in (0, 1):
            dlogits[bounds[2 * pair + side]:bounds[2 * pair + side + 1]] *= slope * weight[side] * loss_scale(case) / case["pairs"]
    return {"loss": torch.tensor(losses, dtype=torch.float64), "logps": logps, "dlogits": dlogits}
