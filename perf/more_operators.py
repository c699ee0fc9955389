"""The operators of fine-tuning next to the selected-token log-probabilities, as cases
to measure: their inputs, their plain forms in elementary torch operations, and their
definitions in 64 bits.

  layer norm       the sum of a residual stream and a block's output, and its layer
                   norm, in one call; and the backward pass with the sums over rows.
  preference loss  the loss of pairs of a chosen and a rejected sequence, from the
                   log-probabilities of their tokens, with its gradient.
  Muon             one step over many matrices: the momentum of each, orthogonalised
                   by Newton-Schulz products.

own = True runs the framework's kernels, own = False the plain forms.
"""

import math
import random

import torch

own = False

DEV = "cuda"
ALIGN = 64  # every matrix starts at a multiple of this in the flat buffers
A, B, C = 3.4445, -4.7750, 2.0315  # a step takes the singular value s to A s + B s^3 + C s^5

FLOAT = {"f32": torch.float32, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "bf16": 2}


# ------------------------------------------------------------------------ cases

def _norm(name, direction, T, d, residual, act, weight, bias, branch, pad=0):
    return {"name": name, "op": "norm", "direction": direction, "T": T, "d": d, "residual": residual, "act": act,
            "weight": weight, "bias": bias, "branch": branch, "pad": pad}


def _preference(name, pairs, shortest, longest, sizes, kind, average, masked, ref, nll, halves):
    return {"name": name, "op": "preference", "pairs": pairs, "shortest": shortest, "longest": longest, "sizes": sizes,
            "kind": kind, "average": average, "masked": masked, "ref": ref, "nll": nll, "halves": halves}


def _muon(name, count, rows, cols, low, sizes, grad, copy, scaling):
    return {"name": name, "op": "muon", "count": count, "rows": rows, "cols": cols, "low": low, "sizes": sizes,
            "grad": grad, "copy": copy, "scaling": scaling}


def listed():
    return [
        # the norm before the LM head when one token is decoded: latency is all there is
        _norm("layer norm one token", "forward", 1, 4096, "bf16", "bf16", "bf16", True, True),
        # the long batch (16384 rows of 2048): a residual stream kept in float32 under bf16 activations
        _norm("layer norm 16384x2048 f32", "forward", 16384, 2048, "f32", "bf16", "f32", True, True),
        # the backward pass of the batch of 512 rows of 4096
        _norm("layer norm back 512x4096", "backward", 512, 4096, "bf16", "bf16", "bf16", True, True),
        # a long batch of wide rows, no bias
        _norm("layer norm back 8192x4096", "backward", 8192, 4096, "bf16", "bf16", "bf16", False, True),
        # odd sizes in float32, rows further apart than they are long
        _norm("layer norm back 1021x2047", "backward", 1021, 2047, "f32", "f32", "f32", True, False, 3),
        # a micro-batch: 4 pairs of answers of up to 64 tokens, no reference
        _preference("preference 4 pairs", 4, 1, 64, 3, "sigmoid", True, 0.0, False, False, False),
        # a large batch: 512 pairs of up to 8192 tokens, prompts masked, a reference, the likelihood term
        _preference("preference 512 pairs", 512, 1, 8192, 4, "sigmoid", False, 0.3, True, True, True),
        # two pairs of long documents: few sequences, many rows
        _preference("preference 2 long pairs", 2, 60000, 131072, 5, "square", True, 0.3, True, False, False),
        # the attention projections of a small model
        _muon("muon 4 x 256x256", 4, 256, 256, 256, 0, "f32", True, "spectral"),
        # one square projection of a model of 4096
        _muon("muon 4096x4096", 1, 4096, 4096, 4096, 0, "bf16", True, "rms"),
        # a small model's matrices of all shapes, wide and tall
        _muon("muon 24 matrices", 24, 2048, 2048, 64, 1, "f32", False, "spectral"),
        # one tall matrix of odd sizes
        _muon("muon 2047x1021", 1, 2047, 1021, 1021, 0, "bf16", False, "spectral"),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["forward", "backward", "preference", "muon"])
    if op in ("forward", "backward"):
        d = _log(rng, 64, 8192)
        d = d if rng.random() < 0.4 else max(64, d // 64 * 64)
        T = _log(rng, 1, min(16384, (1 << 25) // d))
        residual, act = rng.choice([("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32")])
        c = _norm("", op, T, d, residual, act, rng.choice(["bf16", "f32"]), rng.random() < 0.7, rng.random() < 0.7,
                  rng.choice([0, 0, 8, 3]))
    elif op == "preference":
        pairs = _log(rng, 1, 1024)
        longest = _log(rng, 16, min(131072, (1 << 21) // pairs))
        kind = rng.choice(["sigmoid", "sigmoid", "hinge", "square"])
        c = _preference("", pairs, 1, longest, rng.randrange(1 << 20), kind, rng.random() < 0.5,
                        rng.choice([0.0, 0.3, 0.9]), rng.random() < 0.7, rng.random() < 0.3, rng.random() < 0.5)
    else:
        count = rng.choice([1, 1, 1, 2, 5, 16])
        most = int(4096 / count ** (1 / 3))
        rows, cols = _log(rng, 32, most), _log(rng, 32, most)
        if rng.random() < 0.5:
            rows, cols = max(32, rows // 32 * 32), max(32, cols // 32 * 32)
        c = _muon("", count, rows, cols, min(rows, cols, _log(rng, 1, 1024)), rng.randrange(1 << 20),
                  rng.choice(["f32", "bf16"]), rng.random() < 0.5, rng.choice(["spectral", "rms"]))
    del c["name"]
    return c


def _lengths(case):
    """The sequences' lengths, an empty one among many."""
    rng = random.Random(case["sizes"])
    some = [rng.randint(case["shortest"], case["longest"]) for _ in range(2 * case["pairs"])]
    return [0 if i == 11 else n for i, n in enumerate(some)]


def _shapes(case):
    """The matrices' shapes: the largest first, the others spread over the range in logarithm."""
    rng = random.Random(case["sizes"])
    rest = [(_log(rng, case["low"], case["rows"]), _log(rng, case["low"], case["cols"]))
            for _ in range(case["count"] - 1)]
    return [(case["rows"], case["cols"])] + rest


# ------------------------------------------------------------------------ inputs

def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _rows(g, T, d, pad, dtype, scale=1.0):
    """Rows `pad` elements further apart than they are long."""
    return (scale * torch.randn(T, d + pad, generator=g, device=DEV)).to(dtype)[:, :d]


def prepare(case, seed):
    return {"norm": _prepare_norm, "preference": _prepare_preference, "muon": _prepare_muon}[case["op"]](case, _generator(seed))


def _prepare_norm(case, g):
    T, d, pad = case["T"], case["d"], case["pad"]
    act, weight, kind = FLOAT[case["act"]], FLOAT[case["weight"]], FLOAT[case["residual"]]
    s = {"case": case, "eps": 1e-5, "branch": None, "bias": None}
    # a residual stream has a few channels far above the others, and rows whose mean is not zero
    loud = 1 + 20 * (torch.rand(d, generator=g, device=DEV) < 0.01).float()
    s["residual"] = (_rows(g, T, d, pad, torch.float32).mul_(loud) + 0.3).to(kind)
    if case["branch"]:
        s["branch"] = _rows(g, T, d, pad, act, 0.7)
    elif kind != act:  # the norm comes in the stream's type without a branch
        s["residual"] = s["residual"].to(act)
    s["weight"] = (1 + 0.2 * torch.randn(d, generator=g, device=DEV)).to(weight)
    if case["bias"]:
        s["bias"] = (0.2 * torch.randn(d, generator=g, device=DEV)).to(weight)
    if case["direction"] == "backward":
        # what the forward pass kept: the new residual stream, the means and the reciprocal roots
        new, s["mean"], s["rstd"] = _norm_stream(s)
        s["residual"] = new.to(s["residual"].dtype)
        s["grad_normed"] = _rows(g, T, d, pad, act, 1e-2)
        s["grad_residual"] = _rows(g, T, d, pad, s["residual"].dtype, 1e-2)
    return s


def _prepare_preference(case, g):
    lengths = torch.tensor(_lengths(case), device=DEV)
    n = 2 * case["pairs"]
    T = int(lengths.sum())
    cu = torch.zeros(n + 1, dtype=torch.int64, device=DEV)
    cu[1:] = lengths.cumsum(0)
    logp = -torch.empty(T, device=DEV).exponential_(1.0, generator=g)
    s = {"case": case, "cu_seqlens": cu, "T": T, "beta": 2.0 if case["average"] else 0.1, "ref_logp": None, "mask": None,
         "margin": 0.0 if case["ref"] else 0.5, "label_smoothing": 0.1 if case["kind"] == "sigmoid" else 0.0,
         "nll_coef": 0.2 if case["nll"] else 0.0}
    if case["ref"]:
        # the policy has moved by a little in every token
        s["ref_logp"] = logp + torch.randn(T, generator=g, device=DEV) * min(0.3, 10 / math.sqrt(case["longest"]))
    if case["masked"]:
        # a prompt at the start of each sequence, its rows' log-probabilities NaN; one sequence in sixteen has no answer
        place = torch.arange(T, device=DEV) - torch.repeat_interleave(cu[:-1], lengths, output_size=T)
        share = torch.clamp_max(torch.rand(n, generator=g, device=DEV) * 2 * case["masked"], 0.97)
        none = (torch.rand(n, generator=g, device=DEV) < 0.0625) & (torch.arange(n, device=DEV) >= n // 2 + 1)
        share = torch.where(none, torch.ones_like(share), share)
        prompt = torch.repeat_interleave((share * lengths).long(), lengths, output_size=T)
        s["mask"] = place >= prompt
        logp = torch.where(s["mask"], logp, torch.full_like(logp, math.nan))
    s["logp"] = logp
    return s


def _prepare_muon(case, g):
    shapes = _shapes(case)
    at = [0]
    for r, c in shapes:
        at.append(at[-1] + -(-r * c // ALIGN) * ALIGN)
    s = {"case": case, "shapes": shapes, "at": at, "lr": 0.02, "momentum": 0.95, "eps": 1e-7, "weight_decay": 0.1, "steps": 5}
    for name in ("param", "grad", "mom"):
        s[name] = torch.zeros(at[-1], device=DEV)
    s["copy"] = torch.zeros(at[-1], dtype=torch.bfloat16, device=DEV) if case["copy"] else None
    for a, (r, c) in zip(at, shapes):
        # a gradient has a few strong directions over many weak ones, and the momentum shares some of them
        rank = min(8, r, c)
        left = torch.randn(r, rank, generator=g, device=DEV) * 3 ** -torch.arange(rank, device=DEV).float()
        right = torch.randn(rank, c, generator=g, device=DEV)
        noise = 0.1 * torch.randn(2, r, c, generator=g, device=DEV)
        part = slice(a, a + r * c)
        s["param"][part] = 0.02 * torch.randn(r * c, generator=g, device=DEV)
        s["grad"][part] = (1e-3 * (left @ right + noise[0])).view(-1)
        s["mom"][part] = (5e-3 * ((left.flip(0) @ right) + noise[1])).view(-1)
    s["grad"] = s["grad"].to(FLOAT[case["grad"]])
    if own:
        from invariant_token_logprobs_gb300 import tune
        cut = lambda flat: [flat[a:a + r * c].view(r, c) for a, (r, c) in zip(at, shapes)]  # noqa: E731
        s["optimizer"] = tune.Muon(
            cut(s["param"]), cut(s["grad"]), copies=cut(s["copy"]) if case["copy"] else None, lr=s["lr"],
            momentum=s["momentum"], nesterov=True, weight_decay=s["weight_decay"], scaling=case["scaling"], steps=s["steps"],
            eps=s["eps"], state={"momentum": s["mom"]})
    return s


# ------------------------------------------------------------------------ one pass

def run(state):
    op = state["case"]["op"]
    if op == "norm":
        backward = state["case"]["direction"] == "backward"
        if own:
            return _own_norm_backward(state) if backward else _own_norm(state)
        return _plain_norm_backward(state) if backward else _plain_norm(state)
    if op == "preference":
        return _own_preference(state) if own else _plain_preference(state)
    return _own_muon(state) if own else _plain_muon(state)


def _own_norm(s):
    from invariant_token_logprobs_gb300 import tune
    normed, stream, mean, rstd = tune.layer_norm(s["residual"], s["branch"], weight=s["weight"], bias=s["bias"], eps=s["eps"])
    return normed, stream if s["branch"] is not None else None, mean, rstd


def _own_norm_backward(s):
    from invariant_token_logprobs_gb300 import tune
    return tuple(tune.layer_norm_backward(s["grad_normed"], s["grad_residual"], s["residual"], s["mean"], s["rstd"],
                                          weight=s["weight"], bias=s["bias"], branch=s["branch"] is not None))


def _own_preference(s):
    from invariant_token_logprobs_gb300 import tune
    case = s["case"]
    return tuple(tune.preference_loss(s["logp"], s["cu_seqlens"], ref_logp=s["ref_logp"], mask=s["mask"], kind=case["kind"],
                                      beta=s["beta"], margin=s["margin"], label_smoothing=s["label_smoothing"],
                                      average=case["average"], nll_coef=s["nll_coef"], halves=case["halves"]))


def _own_muon(s):
    s["optimizer"].step()
    return s["param"], s["copy"], s["mom"]


# ------------------------------------------------------------------------ plain forms

def _norm_stream(s):
    """The new residual stream in float32, and its rows' means and reciprocal roots."""
    new = s["residual"].float()
    if s["branch"] is not None:
        new = new + s["branch"].float()
    mean = new.mean(1)
    off = new - mean[:, None]
    return new, mean, torch.rsqrt((off * off).mean(1) + s["eps"])


def _plain_norm(s):
    new, mean, rstd = _norm_stream(s)
    normed = (new - mean[:, None]) * rstd[:, None] * s["weight"].float()
    if s["bias"] is not None:
        normed = normed + s["bias"].float()
    if s["branch"] is None:
        return normed.to(s["residual"].dtype), None, mean, rstd
    return normed.to(s["branch"].dtype), new.to(s["residual"].dtype), mean, rstd


def _plain_norm_backward(s):
    dh, x = s["grad_normed"].float(), (s["residual"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    grad_weight = (dh * x).sum(0)
    grad_bias = dh.sum(0) if s["bias"] is not None else None
    dx = dh * s["weight"].float()
    D = s["grad_residual"].float() + s["rstd"][:, None] * (dx - dx.mean(1, keepdim=True) - x * (dx * x).mean(1, keepdim=True))
    grad_branch = D.to(s["grad_normed"].dtype) if s["branch"] is not None else None
    return D.to(s["residual"].dtype), grad_branch, grad_weight, grad_bias


def _plain_preference(s):
    case, T, cu = s["case"], s["T"], s["cu_seqlens"]
    n, P = 2 * case["pairs"], case["pairs"]
    sequence = torch.repeat_interleave(torch.arange(n, device=DEV), cu[1:] - cu[:-1], output_size=T)
    keep = s["mask"] if s["mask"] is not None else torch.ones(T, dtype=torch.bool, device=DEV)
    zero = torch.zeros((), dtype=torch.float64, device=DEV)
    # sums of up to 131072 rows whose difference decides: in 64 bits
    logp = torch.where(keep, s["logp"].double(), zero)
    count = torch.zeros(n, dtype=torch.float64, device=DEV).index_add_(0, sequence, keep.double())
    likely = torch.zeros(n, dtype=torch.float64, device=DEV).index_add_(0, sequence, logp)
    score = likely
    if s["ref_logp"] is not None:
        ref = torch.where(keep, s["ref_logp"].double(), zero)
        score = score - torch.zeros(n, dtype=torch.float64, device=DEV).index_add_(0, sequence, ref)
    each = 1.0 / count.clamp_min(1.0)  # of a row in its sequence's mean
    if case["average"]:
        score = score * each
    pair = (lambda v: v.view(2, P)) if case["halves"] else (lambda v: v.view(P, 2).t())
    counted = (pair(count) > 0).all(0)
    w = counted.double() / counted.double().sum().clamp_min(1.0)
    chosen, rejected = pair(score)
    z = s["beta"] * (chosen - rejected) - s["margin"]
    if case["kind"] == "sigmoid":
        e = s["label_smoothing"]
        up, down = torch.log1p(torch.exp(-z.abs())) + z.clamp_min(0), torch.log1p(torch.exp(-z.abs())) + (-z).clamp_min(0)
        loss, slope = (1 - e) * down + e * up, 1 / (1 + torch.exp(-z)) - (1 - e)
    elif case["kind"] == "hinge":
        loss, slope = (1 - z).clamp_min(0), -(z < 1).double()
    else:
        loss, slope = ((z - 0.5) / s["beta"]).square(), 2 * (z - 0.5) / s["beta"] ** 2
    nll = -(pair(likely)[0] * pair(each)[0])
    preference, likelihood = (w * loss).sum(), (w * nll).sum()
    stats = torch.stack([preference + s["nll_coef"] * likelihood, preference, likelihood,
                         (w * (chosen > rejected).double()).sum(), (w * s["beta"] * chosen).sum(),
                         (w * s["beta"] * rejected).sum()])
    part = pair(each) if case["average"] else torch.ones(2, P, dtype=torch.float64, device=DEV)
    step = w * slope * s["beta"] * part * torch.tensor([[1.0], [-1.0]], dtype=torch.float64, device=DEV)
    step[0] -= w * s["nll_coef"] * pair(each)[0]
    step = step.reshape(-1) if case["halves"] else step.t().reshape(-1)
    grad = torch.where(keep, step.float()[sequence], torch.zeros((), device=DEV))
    return stats.float(), (s["beta"] * score).float(), grad


def _plain_muon(s):
    mu = s["momentum"]
    copy = s["copy"]
    for a, (r, c) in zip(s["at"], s["shapes"]):
        part = slice(a, a + r * c)
        g = s["grad"][part].float()
        m = mu * s["mom"][part] + g
        s["mom"][part] = m
        u = (g + mu * m).view(r, c)
        x = u / (torch.sqrt((u * u).sum()) + s["eps"])
        x = x if r <= c else x.t()
        for _ in range(s["steps"]):
            gram = x @ x.t()
            x = A * x + (B * gram + C * (gram @ gram)) @ x
        x = x if r <= c else x.t()
        scale = math.sqrt(max(1.0, r / c)) if s["case"]["scaling"] == "spectral" else 0.2 * math.sqrt(max(r, c))
        p = s["param"][part].view(r, c) * (1 - s["lr"] * s["weight_decay"]) - (s["lr"] * scale) * x
        s["param"][part] = p.reshape(-1)
        if copy is not None:
            copy[part] = p.reshape(-1).to(torch.bfloat16)
    return s["param"], copy, s["mom"]


# ------------------------------------------------------------------------ work

def work(case):
    if case["op"] == "norm":
        T, d, a, w = case["T"], case["d"], BYTES[case["act"]], BYTES[case["weight"]]
        r = BYTES[case["residual"]] if case["branch"] else a
        vectors = d * w * (1 + case["bias"])
        if case["direction"] == "forward":
            # the stream and the block's output in, the new stream and its norm out; without a block's output one of each
            rows = 2 * (r + a) if case["branch"] else r + a
            return {"bytes": T * d * rows + vectors + 8 * T, "flops": 9 * T * d}
        # the stream and both gradients in, the gradient out (in both types where they differ)
        rows = 3 * r + a + (a if case["branch"] and r != a else 0)
        return {"bytes": T * d * rows + d * w + 4 * d * (1 + case["bias"]) + 8 * T, "flops": 16 * T * d}
    if case["op"] == "preference":
        T, n = sum(_lengths(case)), 2 * case["pairs"]
        each = 8 + (4 if case["ref"] else 0) + (1 if case["masked"] else 0)
        return {"bytes": T * each + 8 * (n + 1) + 4 * n, "flops": 8 * T}
    moved = flops = 0
    for r, c in _shapes(case):
        m, n = min(r, c), max(r, c)
        # gradient in, momentum and parameter in and out
        moved += r * c * (BYTES[case["grad"]] + 16 + (2 if case["copy"] else 0))
        # two of the three products of a step are symmetric: half of each is enough
        flops += 5 * (3 * m * m * n + m * m * m)
    return {"bytes": moved, "flops": flops}


# ------------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "preference": _exact_preference, "muon": _exact_muon}[case["op"]](s)


def _exact_norm(s):
    d = s["case"]["d"]
    w = s["weight"].double()
    if s["case"]["direction"] == "forward":
        new = s["residual"].double() + (0 if s["branch"] is None else s["branch"].double())
        mean = new.sum(1) / d
        rstd = ((new.square().sum(1) / d - mean.square()) + s["eps"]).pow(-0.5)
        normed = torch.addcmul(0 * new if s["bias"] is None else s["bias"].double().expand_as(new),
                               (new - mean[:, None]) * rstd[:, None], w.expand_as(new))
        return normed, None if s["branch"] is None else new, mean, rstd
    # dL/d(new) = dnew + J^T dh, J the derivative of (new - mean) * rstd * w
    mean, rstd, dh = s["mean"].double()[:, None], s["rstd"].double()[:, None], s["grad_normed"].double()
    off = s["residual"].double() - mean
    wdh = w * dh
    dot = (wdh * off).sum(1, keepdim=True)
    D = s["grad_residual"].double() + rstd * wdh - rstd * wdh.sum(1, keepdim=True) / d - off * dot * rstd ** 3 / d
    # the sums over the rows as products
    ones = torch.ones(1, off.shape[0], dtype=torch.float64, device=DEV)
    return (D, None if s["branch"] is None else D, (ones @ (dh * off * rstd))[0],
            None if s["bias"] is None else (ones @ dh)[0])


def _exact_preference(s):
    case, T, cu = s["case"], s["T"], s["cu_seqlens"]
    P, beta = case["pairs"], s["beta"]
    keep = s["mask"] if s["mask"] is not None else torch.ones(T, dtype=torch.bool, device=DEV)
    zero = torch.zeros(1, dtype=torch.float64, device=DEV)

    def sums(v):  # by differences of running sums at the sequences' ends
        run = torch.cat([zero, torch.where(keep, v.double(), zero).cumsum(0)])
        return run[cu[1:]] - run[cu[:-1]]

    count, likely = sums(keep), sums(s["logp"])
    score = likely - (0 if s["ref_logp"] is None else sums(s["ref_logp"]))
    if case["average"]:
        score = torch.where(count > 0, score / count, score)
    first = torch.arange(P, device=DEV) * (1 if case["halves"] else 2)
    second = first + (P if case["halves"] else 1)
    have = (count[first] > 0) & (count[second] > 0)
    c, r = first[have], second[have]
    N = max(1, int(have.sum()))
    gap = beta * (score[c] - score[r]) - s["margin"]
    if case["kind"] == "sigmoid":
        e = s["label_smoothing"]
        ln = torch.nn.functional.logsigmoid
        loss = -(1 - e) * ln(gap) - e * ln(-gap)
        slope = e * torch.sigmoid(gap) - (1 - e) * torch.sigmoid(-gap)
    elif case["kind"] == "hinge":
        loss = torch.where(gap < 1, 1 - gap, 0 * gap)
        slope = torch.where(gap < 1, -torch.ones_like(gap), torch.zeros_like(gap))
    else:
        loss = ((score[c] - score[r]) - (s["margin"] + 0.5) / beta).square()
        slope = 2 * ((score[c] - score[r]) - (s["margin"] + 0.5) / beta) / beta
    nll = -(likely[c] / count[c])
    coefficient = torch.zeros(2 * P, dtype=torch.float64, device=DEV)
    coefficient[c] = (slope * beta / (count[c] if case["average"] else 1) - s["nll_coef"] / count[c]) / N
    coefficient[r] = -(slope * beta / (count[r] if case["average"] else 1)) / N
    at = torch.searchsorted(cu[1:], torch.arange(T, device=DEV), right=True)
    grad = coefficient[at] * keep
    means = [float(v.sum()) / N for v in (loss, nll, score[c] > score[r], beta * score[c], beta * score[r])]
    return torch.tensor([means[0] + s["nll_coef"] * means[1]] + means, dtype=torch.float64), beta * score, grad


def _exact_muon(s):
    param, mom = s["param"].double(), s["mom"].double()
    for a, (r, c) in zip(s["at"], s["shapes"]):
        part = slice(a, a + r * c)
        g = s["grad"][part].double()
        mom[part] = s["momentum"] * mom[part] + g
        x = (s["momentum"] * mom[part] + g).view(r, c)
        x = x / (torch.linalg.vector_norm(x) + s["eps"])
        tall = r > c
        for _ in range(s["steps"]):  # C Z (Z x) + B (Z x) + A x, Z the smaller of the two Gram matrices
            if tall:
                z = x.mT @ x
                y = x @ z
                x = torch.add(A * x + B * y, y @ z, alpha=C)
            else:
                z = x @ x.mT
                y = z @ x
                x = torch.add(A * x + B * y, z @ y, alpha=C)
        scale = max(1.0, r / c) ** 0.5 if s["case"]["scaling"] == "spectral" else 0.2 * max(r, c) ** 0.5
        param[part] -= s["lr"] * (s["weight_decay"] * param[part] + scale * x.reshape(-1))
    return param, param if s["copy"] is not None else None, mom
