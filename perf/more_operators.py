"""What is measured of the draft head in 4 bits and of the scores read from a head's logits: the
quantisation of rows to 4-bit floating point with a scale for every 32 entries, the head's product
over such rows, log-probabilities of given tokens with their rank, the row's entropy and its top
alternatives, and the gradient of log-probability and entropy.

`run` computes the plain form with elementary torch operations; with `own` true it makes the calls a
user makes of the library. Inputs, outputs and their layouts are those of include/spec_mxfp4.h and
include/spec_logprobs.h.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
BLOCK = 32    # entries that share a scale
WHOLE = 128   # a row's entries are padded to a multiple of this


def _sv():
    import device_draft_verification_amd as sv
    return sv


# ------------------------------------------------------------------ cases ---

def listed():
    return [
        # hidden states of a decode batch, with the values that the codes stand for: latency
        dict(name="quantize_hidden", op="quantize", N=64, D=4096, dtype="bf16"),
        # rows of every position of the verification benchmark, of an odd length
        dict(name="quantize_odd", op="quantize", N=2304, D=4001, dtype="f32"),
        # a head's weights in a training step that goes through their 4-bit values
        dict(name="quantize_weights", op="quantize", N=152064, D=4096, dtype="bf16"),
        # one token of one sequence through a small head: latency
        dict(name="head_one", op="head", N=1, D=4096, V=32000, dtype="bf16", out="f32"),
        # an odd vocabulary and a depth that is no multiple of a block
        dict(name="head_odd", op="head", N=37, D=1000, V=20011, dtype="f32", out="f32"),
        # a decode batch through the full head: bound by reading the weights
        dict(name="head_decode", op="head", N=64, D=4096, V=152064, dtype="bf16", out="bf16"),
        # every target row of the verification benchmark: bound by the matrix cores
        dict(name="head_large", op="head", N=2304, D=4096, V=152064, dtype="bf16", out="bf16"),
        # one served token with its top alternatives, logits of a full fp32 head: latency
        dict(name="scores_one", op="scores", N=1, V=128256, K=20, dtype="f32"),
        # the scores of a short prompt, an odd vocabulary (rows not 16-byte aligned)
        dict(name="scores_odd", op="scores", N=37, V=20011, K=5, dtype="bf16"),
        # every target row of the verification benchmark, lists long enough to be a teacher's
        dict(name="scores_large", op="scores", N=2304, V=152064, K=64, dtype="bf16"),
        # a short batch trained on its own tokens: score, entropy and their gradient, fp32 logits
        dict(name="train_small", op="train", N=37, V=20011, dtype="f32"),
        # the same over every target row of the verification benchmark
        dict(name="train_large", op="train", N=2304, V=152064, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantize", "head", "head", "scores", "scores", "train"])
    if op == "quantize":
        D = _log_int(rng, 1, 8192)
        if rng.random() < 0.5:
            D = (D + 31) // 32 * 32
        dtype = rng.choice(["f32", "bf16"])
        room = 152064 * 4096 * 2 // (D * (4 if dtype == "f32" else 2))
        return dict(op=op, N=_log_int(rng, 1, min(152064, room)), D=D, dtype=dtype)
    if op == "head":
        D = _log_int(rng, 32, 4096)
        if rng.random() < 0.7:
            D = (D + 31) // 32 * 32
        V = _log_int(rng, 1000, 152064)
        return dict(op=op, N=_log_int(rng, 1, 2304), D=D, V=V if rng.random() < 0.5 else V // 8 * 8,
                    dtype=rng.choice(["f32", "bf16"]), out=rng.choice(["f32", "bf16", "bf16"]))
    dtype = rng.choice(["f32", "bf16", "bf16"])
    V = _log_int(rng, 1000, 201088)
    if rng.random() < 0.5:
        V = V // 8 * 8
    room = 2304 * 152064 * 2 // (V * (4 if dtype == "f32" else 2))
    c = dict(op=op, N=_log_int(rng, 1, max(1, min(2304, room))), V=V, dtype=dtype)
    if op == "scores":
        c["K"] = _log_int(rng, 1, 64)
    return c


# ----------------------------------------------------------------- inputs ---

def _hidden(n, d, g):
    """Hidden states: a few channels are far larger than the others."""
    x = torch.empty(n, d, device=DEV).normal_(0, 1, generator=g)
    loud = torch.rand(d, device=DEV, generator=g) < 0.01
    return x.mul_(torch.where(loud, 12.0, 1.0))


def _weights(n, d, g):
    """A head's weights, in pieces of rows."""
    for r in range(0, n, 16384):
        yield slice(r, min(n, r + 16384)), torch.empty(
            min(16384, n - r), d, device=DEV).normal_(0, 0.02, generator=g)


def _rows_inputs(c, g):
    N, V = c["N"], c["V"]
    z = torch.empty(N, V, device=DEV).normal_(0, 2.5, generator=g)
    # some rows of a grammar that allows part of the vocabulary, one in fifty of them none
    masked = torch.rand(N, device=DEV, generator=g) < 0.25
    share = torch.rand(N, device=DEV, generator=g).pow_(3)
    none = torch.rand(N, device=DEV, generator=g) < (0.02 if N > 8 else 0.0)
    share = torch.where(masked, share.masked_fill_(none, 0.0), 2.0)
    temperature = torch.where(torch.rand(N, device=DEV, generator=g) < 0.5, 1.0,
                              torch.empty(N, device=DEV).uniform_(0.7, 2.0, generator=g))
    token = torch.empty(N, dtype=torch.int32, device=DEV)
    logits = torch.empty(N, V, dtype=DTYPES[c["dtype"]], device=DEV)
    for n in range(0, N, 256):
        at = slice(n, min(N, n + 256))
        u = torch.rand(z[at].shape, device=DEV, generator=g)
        logits[at] = z[at].masked_fill_(u >= share[at, None], -math.inf).to(logits.dtype)
        # tokens drawn from their rows (the largest of logit over temperature plus Gumbel noise)
        noise = u.exponential_(1.0, generator=g).log_().neg_()
        token[at] = noise.add_(logits[at] / temperature[at, None]).argmax(1)
    # a padded batch has rows without a token, as has a row that its mask leaves empty
    padded = (torch.rand(N, device=DEV, generator=g) < (0.05 if N > 8 else 0.0)) | (share <= 0)
    return dict(logits=logits, token=token.masked_fill_(padded, -1), temperature=temperature)


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op, N = c["op"], c["N"]
    s = dict(case=c)
    if op in ("quantize", "head"):
        D = c["D"]
        whole = (D + WHOLE - 1) // WHOLE * WHOLE
        codes = lambda n: torch.empty(n, whole // 2, dtype=torch.uint8, device=DEV)
        scales = lambda n: torch.empty(n, whole // BLOCK, dtype=torch.uint8, device=DEV)
        s["q"], s["scale"] = codes(N), scales(N)
    if op == "quantize":
        x = torch.empty(N, D, dtype=DTYPES[c["dtype"]], device=DEV)
        if N > 4096:
            for at, w in _weights(N, D, g):
                x[at] = w.to(x.dtype)
        else:
            x.copy_(_hidden(N, D, g))
        s["x"], s["values"] = x, torch.empty_like(x)
    elif op == "head":
        V = c["V"]
        s["x"] = _hidden(N, D, g).to(DTYPES[c["dtype"]])
        s["w"], s["w_scale"] = codes(V), scales(V)
        for at, w in _weights(V, D, g):
            s["w"][at], s["w_scale"][at] = _codes(w)
        s["out"] = torch.empty(N, V, dtype=DTYPES[c["out"]], device=DEV)
    else:
        s.update(_rows_inputs(c, g))
        K = c.get("K", 0)
        f32 = lambda *shape: torch.empty(*shape, device=DEV)
        s["logprob"], s["entropy"], s["norm"] = f32(N), f32(N), f32(N, 2)
        s["rank"] = torch.empty(N, dtype=torch.int32, device=DEV)
        if K:
            s["top_token"], s["top_logprob"] = torch.empty(N, K, dtype=torch.int32, device=DEV), f32(N, K)
        if op == "train":
            # advantages of the tokens, and a bonus on the rows' entropy
            s["grad_logprob"] = f32(N).normal_(0, 1.0 / N, generator=g)
            s["grad_entropy"] = f32(N).uniform_(0.5e-2 / N, 2e-2 / N, generator=g)
            s["grad"] = torch.empty_like(s["logits"])
        if own:  # the handle that holds the workspace of rows read in pieces
            s["ctx"] = _sv().spec_logprobs_init(N, c["V"], K, DTYPES[c["dtype"]])
    return s


# ------------------------------------------------------------- plain forms ---

def _quantize(x):
    """Magnitude codes 0 .. 7 and signs [N, blocks, 32], scale exponents [N, blocks] of x [N, D]:
    a block's scale is 2^(floor(log2 of its largest magnitude) - 2), at least 2^-127; an entry over
    the scale goes to the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6, ties to the even code."""
    N, D = x.shape
    whole = (D + WHOLE - 1) // WHOLE * WHOLE
    x = torch.nn.functional.pad(x.float(), (0, whole - D)).view(N, whole // BLOCK, BLOCK)
    mag = x.abs()
    top = mag.amax(2)
    e = torch.where(top > 0, torch.frexp(top).exponent - 3, -127).clamp_(min=-127)
    y = torch.ldexp(mag, -e[..., None])
    code = (y > 0.25).to(torch.uint8)
    code += y >= 0.75
    code += y > 1.25
    code += y >= 1.75
    code += y > 2.5
    code += y >= 3.5
    code += y > 5
    return code, torch.signbit(x), e


def _codes(x):
    """Two codes to a byte, the first in the low half, and the scales' exponents plus 127."""
    code, sign, e = _quantize(x)
    code = (code + sign.to(torch.uint8) * 8).flatten(1)
    return code[:, 0::2] + code[:, 1::2] * 16, (e + 127).to(torch.uint8)


def _values(q, scale):
    """What codes stand for, in 32 bits: [N, D padded]."""
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], device=q.device)
    code = torch.stack((q & 15, q >> 4), 2).flatten(1)
    v = table[code.int()].view(q.shape[0], -1, BLOCK)
    return torch.ldexp(v, scale.int()[..., None] - 127).flatten(1)


def _plain_quantize(s):
    x = s["x"]
    code, sign, e = _quantize(x)
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=x.device)
    v = torch.ldexp(table[code.int()], e[..., None])
    v = torch.where(sign, -v, v).flatten(1)[:, :x.shape[1]]
    return dict(values=v.to(x.dtype).contiguous(), scale=(e + 127).to(torch.uint8))


def _plain_head(s):
    a = _values(*_codes(s["x"]))
    return (a @ _values(s["w"], s["w_scale"]).t()).to(s["out"].dtype)


def _plain_norm(s):
    """Scaled logits, their exponentials against the row's largest (rows without an entry: 0), that
    largest, and the logarithm of the sum."""
    x = s["logits"].float() * (1.0 / s["temperature"])[:, None]
    top = x.amax(1, keepdim=True)
    some = top > -math.inf
    x = x - torch.where(some, top, 0.0)
    e = x.exp()
    total = e.sum(1, keepdim=True, dtype=torch.float64)
    log_sum = torch.where(some, total, 1.0).log().float()
    return x, e, some, top, torch.where(some, total, 1.0).float(), log_sum


def _plain_scores(s, K):
    """Log-probability and place of the token, the row's entropy, its K largest (equal ones by the
    lower token) and its normaliser."""
    z, token = s["logits"], s["token"]
    x, e, some, top, total, log_sum = _plain_norm(s)
    there = token >= 0
    t = token.clamp(min=0).long()[:, None]
    logprob = torch.where(there[:, None], torch.where(some, x.gather(1, t) - log_sum, -math.inf), 0.0)
    zt = z.gather(1, t)
    lower = torch.arange(z.shape[1], device=z.device)[None, :] < t
    rank = ((z > zt) | ((z == zt) & lower)).sum(1)
    rank = torch.where(there & some[:, 0], rank, -1)
    mean = torch.where(e > 0, e * x, 0.0).sum(1, keepdim=True) / total
    out = dict(logprob=logprob[:, 0], rank=rank.int(), entropy=torch.where(some, log_sum - mean, 0.0)[:, 0],
               norm=torch.cat((top, log_sum), 1))
    if K:
        n = min(K, z.shape[1])
        zf = z.float()
        least = zf.topk(n, dim=1).values[:, -1:]
        more, same = zf > least, zf == least
        taken = (more | (same & (same.cumsum(1) <= n - more.sum(1, keepdim=True)))) & (zf > -math.inf)
        place = torch.arange(z.shape[1], device=z.device)
        first = torch.where(taken, -place, -z.shape[1]).topk(n, dim=1).values.neg()   # by token
        used = first < z.shape[1]
        first = first.clamp(max=z.shape[1] - 1)
        by = zf.gather(1, first).masked_fill(~used, -math.inf).sort(dim=1, descending=True, stable=True).indices
        first, used = first.gather(1, by), used.gather(1, by)
        pad = torch.nn.functional.pad
        out["top_token"] = pad(first.masked_fill(~used, -1).int(), (0, K - n), value=-1)
        out["top_logprob"] = pad((x.gather(1, first) - log_sum).masked_fill(~used, -math.inf), (0, K - n),
                                 value=-math.inf)
    return out


def _plain_train(s):
    """The scores, and the gradient of sum_n (a_n logprob_n + b_n entropy_n):
    (a (1[v = token] - p) - b p (log p + H)) / T."""
    out = _plain_scores(s, 0)
    x, e, some, _, total, log_sum = _plain_norm(s)
    p = e / total
    logp = torch.where(p > 0, x - log_sum, 0.0)
    a = torch.where(s["token"] >= 0, s["grad_logprob"], 0.0)[:, None]
    grad = -p * (a + s["grad_entropy"][:, None] * (logp + out["entropy"][:, None]))
    grad.scatter_add_(1, s["token"].clamp(min=0).long()[:, None], a)
    grad = torch.where(some, grad * (1.0 / s["temperature"])[:, None], 0.0)
    out["grad"] = grad.to(s["logits"].dtype)
    return out


# ------------------------------------------------------------------- calls ---

def run(s):
    c = s["case"]
    op = c["op"]
    if not own:
        if op in ("scores", "train"):
            return _plain_scores(s, c["K"]) if op == "scores" else _plain_train(s)
        return _plain_quantize(s) if op == "quantize" else _plain_head(s)
    sv = _sv()
    if op == "quantize":
        sv.spec_mxfp4_quantize_rows(s["x"], s["q"], s["scale"], s["values"])
        return dict(values=s["values"], scale=s["scale"])
    if op == "head":
        sv.spec_mxfp4_quantize_rows(s["x"], s["q"], s["scale"])
        sv.spec_mxfp4_product(s["q"], s["scale"], s["w"], s["w_scale"], s["out"])
        return s["out"]
    sv.spec_token_logprobs(s["ctx"], s["logits"], s["token"], s["temperature"], s["logprob"], s["rank"],
                           s["entropy"], s.get("top_token"), s.get("top_logprob"), s["norm"])
    out = {k: s[k] for k in ("logprob", "rank", "entropy", "norm")}
    if op == "scores":
        return dict(out, top_token=s["top_token"], top_logprob=s["top_logprob"])
    sv.spec_token_logprobs_backward(s["ctx"], s["logits"], s["token"], s["temperature"], s["norm"],
                                    s["entropy"], s["grad_logprob"], s["grad_entropy"], s["grad"])
    return dict(out, grad=s["grad"])


# ------------------------------------------------------------------- work ---

def work(c):
    op, N = c["op"], c["N"]
    size = 4 if c["dtype"] == "f32" else 2
    if op == "quantize":
        blocks = (c["D"] + BLOCK - 1) // BLOCK
        return dict(bytes=N * (2 * c["D"] * size + 17 * blocks), flops=4 * N * c["D"])
    if op == "head":
        blocks = (c["D"] + BLOCK - 1) // BLOCK
        out = 4 if c["out"] == "f32" else 2
        return dict(bytes=N * c["D"] * size + c["V"] * 17 * blocks + out * N * c["V"],
                    flops=2 * N * c["D"] * c["V"])
    if op == "scores":
        return dict(bytes=N * (c["V"] * size + 28 + 8 * c["K"]), flops=6 * N * c["V"])
    return dict(bytes=N * (2 * c["V"] * size + 36), flops=12 * N * c["V"])


# ----------------------------------------------------------------- in 64 bits ---

def _exact_values(x):
    """The nearest value of three significant levels to an octave: halves up to 2, then whole numbers
    up to 4, then even ones up to 6."""
    N, D = x.shape
    blocks = (D + BLOCK - 1) // BLOCK
    y = torch.zeros(N, blocks * BLOCK, dtype=torch.float64, device=x.device)
    y[:, :D] = x
    y = y.view(N, blocks, BLOCK)
    top = y.abs().max(2).values
    octave = torch.floor(torch.log2(top))
    # the logarithm may round up to a whole number
    octave = torch.where(torch.exp2(octave) > top, octave - 1, octave)
    unit = torch.exp2(torch.clamp(octave - 2, min=-127.0))[..., None]   # of no entry: 2^-127
    y = y / unit
    step = torch.where(y.abs() < 2, 0.5, torch.where(y.abs() < 4, 1.0, 2.0))
    y = torch.clamp(torch.round(y / step) * step, -6.0, 6.0) * unit
    return y.view(N, -1)[:, :D]


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    op, N = case["op"], case["N"]
    f64 = torch.float64
    if op == "quantize":
        values = torch.empty(N, case["D"], dtype=f64, device=DEV)
        for n in range(0, N, 16384):
            values[n:n + 16384] = _exact_values(s["x"][n:n + 16384].to(f64))
        return dict(values=values, scale=None)
    if op == "head":
        D, V = case["D"], case["V"]
        a = _exact_values(s["x"].to(f64))
        del s
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        _hidden(N, D, g)
        out = torch.empty(N, V, dtype=f64, device=DEV)
        for at, w in _weights(V, D, g):
            out[:, at] = a @ _exact_values(w.to(f64)).t().contiguous()
        return out
    V, K = case["V"], case.get("K", 0)
    new = lambda *shape: torch.empty(*shape, dtype=f64, device=DEV)
    out = dict(logprob=new(N), rank=None, entropy=new(N), norm=new(N, 2))
    if op == "scores":
        out.update(top_token=None, top_logprob=new(N, K).fill_(-math.inf))
    else:
        out["grad"] = new(N, V)
    for n in range(0, N, 256):
        at = slice(n, min(N, n + 256))
        inv = 1.0 / s["temperature"][at]                                 # fp32, as the definition scales
        x = (s["logits"][at].float() * inv[:, None]).to(f64)
        top = x.max(1).values
        empty = torch.isneginf(top)
        lse = torch.logsumexp(x, 1)
        logp = x - torch.where(empty, 0.0, lse)[:, None]
        p = torch.exp(logp)
        token = s["token"][at].long()
        given = token >= 0
        index = torch.where(given, token, 0)[:, None]
        out["logprob"][at] = torch.where(given, logp.gather(1, index)[:, 0], 0.0)
        entropy = torch.special.entr(p).sum(1)
        out["entropy"][at] = entropy
        out["norm"][at] = torch.stack((top, torch.where(empty, 0.0, lse - torch.where(empty, 0.0, top))), 1)
        if op == "scores":
            best = torch.topk(logp, min(K, V), dim=1).values
            out["top_logprob"][at, :best.shape[1]] = best
            continue
        one = torch.zeros_like(p).scatter_(1, index, given.to(f64)[:, None])
        a, b = s["grad_logprob"][at].to(f64)[:, None], s["grad_entropy"][at].to(f64)[:, None]
        d = a * (one - given.to(f64)[:, None] * p) + b * (torch.special.entr(p) - p * entropy[:, None])
        out["grad"][at] = torch.where(empty[:, None], 0.0, d * inv.to(f64)[:, None])
    return out
