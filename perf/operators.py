"""What is measured of the draft side's vocabulary operators: beam selection with the reordering of
the beams' states, distillation from a teacher's top logits with its gradient, and the 8-bit
quantisation of rows with the integer product that reads it.

`run` computes the plain form with elementary torch operations; with `own` true it makes the calls a
user makes of the library. Inputs, outputs and their layouts are those of include/spec_beam.h,
include/spec_distill.h and include/spec_int8.h.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _sv():
    import device_draft_verification_amd as sv
    return sv


# ------------------------------------------------------------------ cases ---

def listed():
    return [
        # one sequence growing a small draft tree, logits of a full fp32 head: latency
        dict(name="beam_one_sequence", op="beam", B=1, W=4, K=4, V=32000, dtype="f32", lse=False),
        # an odd vocabulary (rows not 16-byte aligned), odd beam counts, some beams dead
        dict(name="beam_odd", op="beam", B=3, W=5, K=7, V=20011, dtype="bf16", lse=False),
        # a serving batch, wide trees; the head has returned the normalisers
        dict(name="beam_wide", op="beam", B=64, W=16, K=32, V=128256, dtype="bf16", lse=True),
        # the largest batch of the verification benchmark
        dict(name="beam_large", op="beam", B=256, W=8, K=8, V=152064, dtype="bf16", lse=True),
        # a few recurrent states of one sequence, reordered in place: latency
        dict(name="reorder_small", op="reorder", L=4, B=1, W=4, K=4, S=16384, in_place=True),
        # the key-value prefixes of a batch, copied into the other half of a double buffer
        dict(name="reorder_large", op="reorder", L=8, B=32, W=8, K=8, S=524288, in_place=False),
        # loss and gradient of a short batch, fp32 logits, rows of several list lengths
        dict(name="distill_small", op="distill", N=37, V=20011, K=10, dtype="f32", full=False, calls=2),
        # a step with autograd between the two passes; the teacher's full normaliser is known
        dict(name="distill_two_calls", op="distill", N=640, V=128256, K=32, dtype="bf16", full=True, calls=2),
        # every target row of the verification benchmark, loss and gradient in one call
        dict(name="distill_large", op="distill", N=2304, V=152064, K=64, dtype="bf16", full=False, calls=1),
        # hidden states of the same rows, quantised on their way into the product
        dict(name="quantize_rows", op="quantize", N=2304, D=4096, dtype="bf16"),
        # second factor of the low-rank head for a decode batch: bound by reading the weights
        dict(name="int8_decode", op="int8", N=64, D=512, V=152064, out="bf16"),
        # the full head over every target row: bound by the matrix cores
        dict(name="int8_large", op="int8", N=2304, D=4096, V=152064, out="bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["beam", "beam", "reorder", "distill", "distill", "quantize", "int8"])
    if op == "beam":
        dtype = rng.choice(["f32", "bf16", "bf16"])
        V = _log_int(rng, 1000, 160000)
        if rng.random() < 0.5:
            V = V // 8 * 8
        W, K = rng.randint(1, 16), _log_int(rng, 1, 32)
        room = 256 * 8 * 152064 * 2 // (V * W * (4 if dtype == "f32" else 2))
        B = _log_int(rng, 1, max(1, min(256, room)))
        # where the call forms the normalisers itself, the order of two beams' tokens is settled
        # only down to the normalisers' own rounding: few pairs keep such a draw out of the way
        return dict(op="beam", B=B, W=W, K=K, V=V, dtype=dtype, lse=B * K > 32 or rng.random() < 0.5)
    if op == "reorder":
        L, B, W = rng.randint(1, 16), _log_int(rng, 1, 64), rng.randint(2, 16)
        in_place = rng.random() < 0.5
        K = W if in_place else rng.randint(1, 16)
        most = max(256, min(1 << 20, 8 * 32 * 8 * 524288 // (L * B * max(W, K))))
        return dict(op="reorder", L=L, B=B, W=W, K=K, S=_log_int(rng, 256, most) // 16 * 16,
                    in_place=in_place)
    if op == "distill":
        dtype = rng.choice(["f32", "bf16", "bf16"])
        V = _log_int(rng, 1000, 160000)
        if rng.random() < 0.5:
            V = V // 8 * 8
        room = 2304 * 152064 * 2 // (V * (4 if dtype == "f32" else 2))
        return dict(op="distill", N=_log_int(rng, 1, max(1, min(2304, room))), V=V,
                    K=_log_int(rng, 1, 64), dtype=dtype, full=rng.random() < 0.5,
                    calls=rng.choice([1, 2]))
    if op == "quantize":
        D = _log_int(rng, 64, 8192)
        if rng.random() < 0.7:
            D = (D + 63) // 64 * 64
        return dict(op="quantize", N=_log_int(rng, 1, 4096), D=D, dtype=rng.choice(["f32", "bf16"]))
    D = _log_int(rng, 64, 4096) // 16 * 16
    V = _log_int(rng, 1000, 152064)
    return dict(op="int8", N=_log_int(rng, 1, 2304), D=D, V=V if rng.random() < 0.5 else V // 8 * 8,
                out=rng.choice(["f32", "bf16", "bf16"]))


# ----------------------------------------------------------------- inputs ---

def _beam_inputs(c, g):
    B, W, V = c["B"], c["W"], c["V"]
    logits = torch.empty(B, W, V, device=DEV).normal_(0, 2.5, generator=g).to(DTYPES[c["dtype"]])
    # scores of beams some tokens deep, best first; some sequences have dead beams at the end
    scores = -torch.empty(B, W, device=DEV).exponential_(0.7, generator=g).cumsum(1)
    alive = torch.randint(1, W + 1, (B, 1), device=DEV, generator=g)
    ragged = torch.rand(B, 1, device=DEV, generator=g) < 0.25
    dead = ragged & (torch.arange(W, device=DEV) >= alive)
    scores = scores.masked_fill(dead, -math.inf)
    lse = None
    if c["lse"]:
        lse = torch.empty(B, W, dtype=torch.float64, device=DEV)
        for b in range(0, B, 32):
            lse[b:b + 32] = torch.logsumexp(logits[b:b + 32].double(), -1)
    return dict(logits=logits, scores=scores, lse=lse)


def _distill_inputs(c, g):
    N, V, K = c["N"], c["V"], min(c["K"], c["V"])
    dtype = DTYPES[c["dtype"]]
    z = torch.empty(N, V, device=DEV).normal_(0, 2.5, generator=g)
    # a teacher correlated with the student, of which only the top of each row is kept
    t = torch.empty(N, V, device=DEV).normal_(0, 1.5, generator=g).add_(z, alpha=0.8)
    temperature = torch.empty(N, device=DEV).uniform_(0.7, 2.0, generator=g)
    top, ids = t.topk(K, dim=1)
    lse = None
    if c["full"]:
        lse = torch.empty(N, dtype=torch.float64, device=DEV)
        for n in range(0, N, 256):
            inv = (1.0 / temperature[n:n + 256])[:, None]
            lse[n:n + 256] = torch.logsumexp((t[n:n + 256] * inv).double(), -1)
    del t
    # lists of several lengths, and rows of a padded batch with no list at all
    length = torch.randint(1, K + 1, (N, 1), device=DEV, generator=g)
    ragged = torch.rand(N, 1, device=DEV, generator=g) < 0.25
    empty = torch.rand(N, 1, device=DEV, generator=g) < (0.05 if N > 8 else 0.0)
    unused = (ragged & (torch.arange(K, device=DEV) >= length)) | empty
    ids = ids.to(torch.int32).masked_fill(unused, -1).contiguous()
    weight = torch.empty(N, device=DEV).uniform_(0.5, 1.5, generator=g) / N
    return dict(logits=z.to(dtype), ids=ids, top=top.contiguous(), teacher_lse=lse,
                temperature=temperature, weight=weight)


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op = c["op"]
    s = dict(case=c)
    if op == "beam":
        s.update(_beam_inputs(c, g))
        B, K = c["B"], c["K"]
        s["parent"] = torch.empty(B, K, dtype=torch.int32, device=DEV)
        s["token"] = torch.empty(B, K, dtype=torch.int32, device=DEV)
        s["score"] = torch.empty(B, K, device=DEV)
        s["logq"] = torch.empty(B, K, device=DEV)
        if own:  # the handle that holds the selection's workspace
            s["ctx"] = _sv().spec_beam_init(B, c["W"], K, c["V"], DTYPES[c["dtype"]])
    elif op == "reorder":
        L, B, W, K, S = c["L"], c["B"], c["W"], c["K"], c["S"]
        # finite values of 16 bits, so that equal means equal bit for bit
        state = lambda beams: torch.randint(-30000, 30000, (L, B, beams, S // 2), device=DEV,
                                            generator=g, dtype=torch.int16)
        s["src"] = state(W)
        s["dst"] = s["src"] if c["in_place"] else state(K)
        parent = torch.randint(0, W, (B, K), device=DEV, generator=g, dtype=torch.int32)
        # most first beams go on from themselves; a few slots hold no beam
        parent[:, 0] = 0
        s["parent"] = parent.masked_fill(torch.rand(B, K, device=DEV, generator=g) < 0.05, -1)
    elif op == "distill":
        s.update(_distill_inputs(c, g))
        N = c["N"]
        s["loss"] = torch.empty(N, device=DEV)
        s["lse"] = torch.empty(N, dtype=torch.float64, device=DEV)
        s["grad"] = torch.empty_like(s["logits"])
    elif op == "quantize":
        x = torch.empty(c["N"], c["D"], device=DEV).normal_(0, 1, generator=g)
        # a few channels of hidden states are far larger than the others
        loud = torch.rand(c["D"], device=DEV, generator=g) < 0.01
        x = x * torch.where(loud, 12.0, 1.0)
        s["x"] = x.to(DTYPES[c["dtype"]])
        s["q"] = torch.empty(c["N"], c["D"], dtype=torch.int8, device=DEV)
        s["scale"] = torch.empty(c["N"], device=DEV)
    else:
        ints = lambda n, d: torch.empty(n, d, device=DEV).normal_(
            0, 32, generator=g).round_().clamp_(-127, 127).to(torch.int8)
        s["a"], s["w"] = ints(c["N"], c["D"]), ints(c["V"], c["D"])
        s["a_scale"] = torch.empty(c["N"], device=DEV).uniform_(0.01, 0.05, generator=g)
        s["w_scale"] = torch.empty(c["V"], device=DEV).uniform_(0.0005, 0.002, generator=g)
        s["out"] = torch.empty(c["N"], c["V"], dtype=DTYPES[c["out"]], device=DEV)
    return s


# ------------------------------------------------------------- plain forms ---

def _plain_beam(s):
    """The K largest of score + (logit - normaliser) over a sequence's beams and tokens, equal values
    by the lower beam and token. In 64 bits: whether one candidate is before another is a border."""
    c = s["case"]
    B, W, K, V = c["B"], c["W"], c["K"], c["V"]
    z = s["logits"].double()
    lse = s["lse"]
    if lse is None:
        m = z.amax(-1, keepdim=True)
        lse = (m + (z - m).exp().sum(-1, keepdim=True).log()).squeeze(-1)
    logq = z.sub_(lse[..., None])
    value = (s["scores"].double()[..., None] + logq).view(B, W * V)
    n = min(K, W * V)
    least = value.topk(n, dim=1).values[:, -1:]          # the K-th largest value
    more, same = value > least, value == least
    room = n - more.sum(1, keepdim=True)                 # how many of the equal ones still fit
    taken = (more | (same & (same.cumsum(1) <= room))) & (value > -math.inf)
    place = torch.arange(W * V, device=value.device)
    first = torch.where(taken, -place, -W * V).topk(n, dim=1).values.neg()   # by place
    there = first < W * V
    first = first.clamp(max=W * V - 1)
    v = value.gather(1, first).masked_fill(~there, -math.inf)
    v, by = v.sort(dim=1, descending=True, stable=True)
    first, there = first.gather(1, by), there.gather(1, by)
    q = logq.view(B, W * V).gather(1, first).masked_fill(~there, -math.inf)
    out = dict(parent=(first // V).masked_fill(~there, -1).int(),
               token=(first % V).masked_fill(~there, -1).int(), score=v.float(), logq=q.float())
    if n < K:
        out = {k: torch.nn.functional.pad(t, (0, K - n), value=-1 if k in ("parent", "token") else -math.inf)
               for k, t in out.items()}
    return out


def _plain_reorder(s):
    parent, src, dst = s["parent"], s["src"], s["dst"]
    L, B, W, S = src.shape
    row = torch.arange(B, device=src.device)[:, None] * W + parent.clamp(min=0)
    new = src.view(L, B * W, S).index_select(1, row.view(-1)).view(L, B, -1, S)
    dst.copy_(torch.where((parent < 0)[None, :, :, None], dst, new))
    return dst


def _plain_distill(s):
    """loss = sum_j p_j (log p_j - log q_j) over the list, gradient = weight / T (P q - p)."""
    N, V = s["logits"].shape
    inv = (1.0 / s["temperature"])[:, None]
    x = s["logits"].float() * inv
    used = s["ids"] >= 0
    some = used.any(1, keepdim=True)
    ids = s["ids"].clamp(min=0).long()
    y = (s["top"] * inv).double().masked_fill(~used, -math.inf)
    if s["teacher_lse"] is None:
        m = y.amax(1, keepdim=True)
        m = torch.where(some, m, 0.0)
        total = (y - m).exp().sum(1, keepdim=True)
        logp = y - (m + torch.where(some, total, 1.0).log())
    else:
        logp = y - s["teacher_lse"][:, None]
    p = logp.exp()
    m = x.amax(1, keepdim=True)
    e = (x - m).exp()
    total = e.sum(1, keepdim=True)
    lse = m.double() + total.double().log()
    logq = x.gather(1, ids).double() - lse
    loss = torch.where(used, p * (logp - logq), 0.0).sum(1)
    scale = s["weight"][:, None] * inv * p.sum(1, keepdim=True).float()
    grad = e.mul_(scale / total)
    grad.scatter_add_(1, ids, torch.where(used, -(p * s["weight"][:, None] * inv), 0.0).float())
    return dict(loss=loss.float(), grad=grad.to(s["logits"].dtype))


def _plain_quantize(s):
    x = s["x"].float()
    # both quotients decide roundings: in 64 bits, the scale then rounded to 32 once
    scale = (x.abs().amax(1).double() / 127).float()
    q = (x.double() / scale.double()[:, None]).round().clamp(-127, 127)
    q = torch.where(scale[:, None] > 0, q, 0.0)
    return dict(q=q.to(torch.int8), scale=scale)


def _plain_int8(s):
    acc = s["a"].float() @ s["w"].float().t()
    z = acc.mul_(s["a_scale"][:, None]).mul_(s["w_scale"][None, :])
    return z.to(s["out"].dtype)


# ------------------------------------------------------------------- calls ---

def run(s):
    c = s["case"]
    op = c["op"]
    if not own:
        return {"beam": _plain_beam, "reorder": _plain_reorder, "distill": _plain_distill,
                "quantize": _plain_quantize, "int8": _plain_int8}[op](s)
    sv = _sv()
    if op == "beam":
        sv.spec_beam_select(s["ctx"], s["logits"], s["scores"], s["lse"], s["parent"], s["token"],
                            s["score"], s["logq"])
        return {k: s[k] for k in ("parent", "token", "score", "logq")}
    if op == "reorder":
        sv.spec_beam_reorder(s["parent"], s["src"], s["dst"])
        return s["dst"]
    if op == "distill":
        if c["calls"] == 1:
            sv.spec_distill_loss_grad(s["logits"], s["ids"], s["top"], s["teacher_lse"],
                                      s["temperature"], s["weight"], s["loss"], s["lse"], s["grad"])
        else:
            sv.spec_distill_forward(s["logits"], s["ids"], s["top"], s["teacher_lse"],
                                    s["temperature"], s["loss"], s["lse"])
            sv.spec_distill_backward(s["logits"], s["ids"], s["top"], s["teacher_lse"],
                                     s["temperature"], s["lse"], s["weight"], s["grad"])
        return {k: s[k] for k in ("loss", "grad")}
    if op == "quantize":
        sv.spec_quantize_rows(s["x"], s["q"], s["scale"])
        return {k: s[k] for k in ("q", "scale")}
    sv.spec_int8_product(s["a"], s["a_scale"], s["w"], s["w_scale"], s["out"])
    return s["out"]


# ------------------------------------------------------------------- work ---

def work(c):
    op = c["op"]
    if op == "beam":
        rows = c["B"] * c["W"]
        size = 4 if c["dtype"] == "f32" else 2
        return dict(bytes=rows * (c["V"] * size + 4 + (8 if c["lse"] else 0)) + 16 * c["B"] * c["K"],
                    flops=rows * c["V"] * (1 if c["lse"] else 4))
    if op == "reorder":
        return dict(bytes=2 * c["L"] * c["B"] * c["K"] * c["S"], flops=0)
    if op == "distill":
        size = 4 if c["dtype"] == "f32" else 2
        return dict(bytes=c["N"] * (2 * c["V"] * size + 8 * c["K"] + 20), flops=8 * c["N"] * c["V"])
    if op == "quantize":
        size = 4 if c["dtype"] == "f32" else 2
        return dict(bytes=c["N"] * (c["D"] * (size + 1) + 4), flops=4 * c["N"] * c["D"])
    size = 4 if c["out"] == "f32" else 2
    return dict(bytes=c["D"] * (c["N"] + c["V"]) + 4 * (c["N"] + c["V"]) + size * c["N"] * c["V"],
                flops=2 * c["N"] * c["D"] * c["V"])


# ----------------------------------------------------------------- in 64 bits ---

def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    op = case["op"]
    f64 = torch.float64
    if op == "beam":
        B, W, K, V = case["B"], case["W"], case["K"], case["V"]
        score = torch.full((B, K), -math.inf, dtype=f64, device=DEV)
        logq = torch.full((B, K), -math.inf, dtype=f64, device=DEV)
        for b in range(B):
            lp = s["logits"][b].to(f64)
            lp = lp - (torch.logsumexp(lp, -1) if s["lse"] is None else s["lse"][b])[:, None]
            flat = (lp + s["scores"][b].to(f64)[:, None]).flatten()
            order = torch.sort(flat, descending=True, stable=True).indices[:K]
            order = order[flat[order] > -math.inf]
            score[b, :order.numel()] = flat[order]
            logq[b, :order.numel()] = lp.flatten()[order]
        return dict(parent=None, token=None, score=score, logq=logq)
    if op == "reorder":
        return None
    if op == "distill":
        N, V = s["logits"].shape
        loss = torch.zeros(N, dtype=f64, device=DEV)
        grad = torch.empty(N, V, dtype=f64, device=DEV)
        step = 256
        for n in range(0, N, step):
            at = slice(n, min(N, n + step))
            inv = (1.0 / s["temperature"][at])[:, None]              # fp32, as the definition scales
            log_student = torch.log_softmax((s["logits"][at].float() * inv).to(f64), -1)
            valid = s["ids"][at] != -1
            index = torch.where(valid, s["ids"][at], 0).long()
            y = torch.where(valid, (s["top"][at] * inv).to(f64), -math.inf)
            norm = torch.logsumexp(y, 1) if s["teacher_lse"] is None else s["teacher_lse"][at]
            norm = torch.where(valid.any(1), norm, 0.0)
            log_teacher = y - norm[:, None]
            teacher = torch.exp(log_teacher)
            diff = log_teacher - log_student.gather(1, index)
            loss[at] = torch.where(teacher > 0, teacher * diff, 0.0).sum(1)
            dense = torch.zeros_like(log_student).scatter_add_(1, index, teacher)
            d = torch.exp(log_student) * teacher.sum(1, keepdim=True) - dense
            grad[at] = d * (s["weight"][at].to(f64)[:, None] * inv.to(f64))
        return dict(loss=loss, grad=grad)
    if op == "quantize":
        top = s["x"].to(f64).abs().max(1).values
        return dict(q=None, scale=top / 127)
    out = torch.empty(case["N"], case["V"], dtype=f64, device=DEV)
    a = s["a"].to(f64) * s["a_scale"].to(f64)[:, None]
    for v in range(0, case["V"], 16384):
        w = s["w"][v:v + 16384].to(f64) * s["w_scale"][v:v + 16384].to(f64)[:, None]
        out[:, v:v + 16384] = a @ w.t().contiguous()
    return out
