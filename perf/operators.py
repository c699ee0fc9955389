"""The operators of a training step next to the selected-token log-probabilities,
as cases to measure: their inputs, their plain forms in elementary torch
operations, and their definitions in 64 bits.

  residual norm   the norm of a block's output, its gate and residual scale, and the
                  norm of the new residual stream that feeds the next block or the
                  LM head, in one call; and its backward pass.
  AdamW           one step over many tensors at once, moments in 32 bits or in 8.
  policy loss     the clipped policy-gradient loss of the selected tokens'
                  log-probabilities, with its gradients.

own = True runs the framework's kernels, own = False the plain forms.
"""

import math
import random

import torch

own = False

DEV = "cuda"
ALIGN = 2048  # every tensor of an optimizer starts at a multiple of this in its flat buffers
BLOCK = 256   # elements that share a scale in 8-bit moments

FLOAT = {"f32": torch.float32, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "bf16": 2}


# ------------------------------------------------------------------------ cases

def _norm(name, direction, T, d, residual, act, weight, post, gate, pad=0):
    return {"name": name, "op": "norm", "direction": direction, "T": T, "d": d, "residual": residual, "act": act,
            "weight": weight, "post": post, "gate": gate, "pad": pad}


def _adamw(name, bits, grad, count, low, high, sizes, copy, clip, step):
    return {"name": name, "op": "adamw", "bits": bits, "grad": grad, "count": count, "low": low, "high": high,
            "sizes": sizes, "copy": copy, "clip": clip, "step": step}


def _policy(name, sequences, longest, sizes, reduction, per_sequence, masked, ref, entropy):
    return {"name": name, "op": "policy", "sequences": sequences, "longest": longest, "sizes": sizes,
            "reduction": reduction, "per_sequence": per_sequence, "masked": masked, "ref": ref, "entropy": entropy}


def listed():
    return [
        # the norm before the LM head when one token is decoded: latency is all there is
        _norm("norm one token", "forward", 1, 4096, "bf16", "bf16", "bf16", False, "none"),
        # the batch of the fused headline (512 rows of 4096): a block's output normed, gated by channel, added
        _norm("norm 512x4096 gated", "forward", 512, 4096, "bf16", "bf16", "bf16", True, "channel"),
        # the long batch (16384 rows of 2048): a residual stream kept in float32 under bf16 activations
        _norm("norm 16384x2048 f32 stream", "forward", 16384, 2048, "f32", "bf16", "f32", True, "none"),
        # the backward pass of the headline batch
        _norm("norm backward 512x4096 gated", "backward", 512, 4096, "bf16", "bf16", "bf16", True, "channel"),
        # a long batch of wide rows through the common pre-norm block: one norm, no gate
        _norm("norm backward 8192x4096", "backward", 8192, 4096, "bf16", "bf16", "bf16", False, "none"),
        # odd sizes in float32 with a gate for every token, rows further apart than they are long
        _norm("norm backward 1021x2047 odd", "backward", 1021, 2047, "f32", "f32", "f32", True, "token", 3),
        # the LM head of 151936 x 4096 and its norm: fp32 main gradients, the bf16 weights written too
        _adamw("adamw head 32 bit", 32, "f32", 2, 4096, 151936 * 4096, 0, True, False, 1000),
        # the head of 151936 x 2048 with 8-bit moments and bf16 gradients
        _adamw("adamw head 8 bit", 8, "bf16", 2, 2048, 151936 * 2048, 0, True, False, 1000),
        # 300 tensors of all sizes, clipped by their global norm
        _adamw("adamw 300 tensors clipped", 32, "f32", 300, 64, 1 << 22, 1, False, True, 10),
        # a small head (8192 x 256) and odd small tensors around it on their first step, 8-bit moments
        _adamw("adamw small 8 bit", 8, "f32", 12, 63, 8192 * 256, 2, True, False, 0),
        # 8 sequences of up to 64 tokens: a micro-batch of 512 rows at most
        _policy("policy small", 8, 64, 3, "token", False, 0.3, False, True),
        # a rollout batch: 1024 ragged sequences of up to 8192 tokens, prompts masked, a reference policy
        _policy("policy rollout", 1024, 8192, 4, "sequence", True, 0.3, True, True),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["forward", "backward", "adamw", "policy"])
    if op in ("forward", "backward"):
        d = _log(rng, 64, 8192)
        d = d if rng.random() < 0.4 else max(64, d // 64 * 64)
        T = _log(rng, 1, min(16384, (1 << 25) // d))
        residual, act = rng.choice([("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32")])
        c = _norm("", op, T, d, residual, act, rng.choice(["bf16", "f32"]), rng.random() < 0.5,
                  rng.choice(["none", "channel", "token"]), rng.choice([0, 0, 8, 3]))
    elif op == "adamw":
        count = _log(rng, 1, 300)
        high = max(64, min(1 << 26, (1 << 28) // count))
        c = _adamw("", rng.choice([32, 8]), rng.choice(["f32", "bf16"]), count, _log(rng, 1, 64), _log(rng, 64, high),
                   rng.randrange(1 << 20), rng.random() < 0.5, False, rng.choice([0, 1, 100, 10000]))
        c["clip"] = c["bits"] == 32 and rng.random() < 0.5
    else:
        sequences = _log(rng, 1, 2048)
        c = _policy("", sequences, _log(rng, 16, min(16384, (1 << 22) // sequences)), rng.randrange(1 << 20),
                    rng.choice(["token", "sequence"]), rng.random() < 0.5, rng.choice([0.0, 0.3, 0.9]),
                    rng.random() < 0.5, rng.random() < 0.7)
    del c["name"]
    return c


def _sizes(case):
    """The tensors' element counts: the largest first, the others spread over the range in logarithm."""
    rng = random.Random(case["sizes"])
    rest = [_log(rng, case["low"], case["high"]) for _ in range(case["count"] - 2)]
    return ([case["high"]] + rest + [case["low"]])[:case["count"]]


def _lengths(case):
    """The sequences' lengths, an empty one among many."""
    rng = random.Random(case["sizes"])
    some = [rng.randint(1, case["longest"]) for _ in range(case["sequences"])]
    return [0 if i == 5 else n for i, n in enumerate(some)]


# ------------------------------------------------------------------------ inputs

def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _rows(g, T, d, pad, dtype, scale=1.0):
    """Rows `pad` elements further apart than they are long."""
    return (scale * torch.randn(T, d + pad, generator=g, device=DEV)).to(dtype)[:, :d]


def prepare(case, seed):
    return {"norm": _prepare_norm, "adamw": _prepare_adamw, "policy": _prepare_policy}[case["op"]](case, _generator(seed))


def _prepare_norm(case, g):
    T, d, pad = case["T"], case["d"], case["pad"]
    act, weight = FLOAT[case["act"]], FLOAT[case["weight"]]
    s = {"case": case, "residual_scale": 1.0, "branch_scale": 0.5, "eps": 1e-6}
    # a residual stream has a few channels far above the others
    loud = 1 + 20 * (torch.rand(d, generator=g, device=DEV) < 0.01).float()
    s["residual"] = _rows(g, T, d, pad, torch.float32).mul_(loud).to(FLOAT[case["residual"]])
    s["branch"] = _rows(g, T, d, pad, act, 0.7)
    s["weight"] = (1 + 0.2 * torch.randn(d, generator=g, device=DEV)).to(weight)
    s["branch_weight"] = (1 + 0.2 * torch.randn(d, generator=g, device=DEV)).to(weight) if case["post"] else None
    s["gate"] = None
    if case["gate"] == "channel":
        s["gate"] = (0.3 * torch.randn(d, generator=g, device=DEV)).to(act)
    elif case["gate"] == "token":
        s["gate"] = _rows(g, T, d, pad, act, 0.3)
    if case["direction"] == "backward":
        # what the forward pass kept: the new residual stream and both norms' reciprocal roots
        new, rstd, branch_rstd = _norm_stream(s)
        s["residual"], s["rstd"], s["branch_rstd"] = new.to(FLOAT[case["residual"]]), rstd, branch_rstd
        s["grad_normed"] = _rows(g, T, d, pad, act, 1e-2)
        s["grad_residual"] = _rows(g, T, d, pad, FLOAT[case["residual"]], 1e-2)
    return s


def _flat(sizes):
    """Where each tensor starts in a flat buffer, and the buffer's length."""
    at = [0]
    for n in sizes:
        at.append(at[-1] + -(-n // ALIGN) * ALIGN)
    return at


def _prepare_adamw(case, g):
    sizes = _sizes(case)
    at = _flat(sizes)
    total = at[-1]
    inside = torch.zeros(total, dtype=torch.bool, device=DEV)
    for a, n in zip(at, sizes):
        inside[a:a + n] = True
    # gradients of a row are alike in size, and rows differ by orders of magnitude
    size = torch.exp(1.5 * torch.randn(total // ALIGN, 1, generator=g, device=DEV)).mul_(1e-3)

    def filled(scale=1.0):
        return torch.randn(total, generator=g, device=DEV).mul_(scale).mul_(inside)

    s = {"case": case, "sizes": sizes, "at": at, "step": case["step"], "lr": 1e-3, "betas": (0.9, 0.99), "eps": 1e-8,
         "seed": 17, "max_norm": 1.0 if case["clip"] else None}
    s["param"] = filled(0.02)
    s["grad"] = filled().view(-1, ALIGN).mul_(size).view(-1).to(FLOAT[case["grad"]])
    s["copy"] = torch.zeros(total, dtype=torch.bfloat16, device=DEV) if case["copy"] else None
    # matrices decay, vectors of up to 8192 do not
    s["weight_decay"] = [0.1 if n > 8192 else 0.0 for n in sizes]
    # the same for each row of ALIGN elements
    rows = torch.tensor([(b - a) // ALIGN for a, b in zip(at[:-1], at[1:])], device=DEV)
    s["decay_rows"] = torch.repeat_interleave(torch.tensor(s["weight_decay"], device=DEV), rows)[:, None]
    started = float(case["step"] > 0)
    m = filled(0.3 * started).view(-1, ALIGN).mul_(size).view(-1)
    v = filled(started).view(-1, ALIGN).mul_(size).view(-1)
    v = v * v * 0.5 + (0.3 * m * m)
    if case["bits"] == 8:
        half = torch.full((1,), 1 << 15, dtype=torch.int64, device=DEV)
        s["m"], s["m_scale"] = _encode(m, True, half)
        s["v"], s["v_scale"] = _encode(torch.sqrt(v), False, half)
    else:
        s["m"], s["v"], s["m_scale"], s["v_scale"] = m, v, None, None
    if own:
        from invariant_token_logprobs_gb300 import train
        cut = lambda flat: [flat[a:a + n] for a, n in zip(at, sizes)]  # noqa: E731
        s["optimizer"] = train.AdamW(
            cut(s["param"]), cut(s["grad"]), copies=cut(s["copy"]) if case["copy"] else None, lr=s["lr"], betas=s["betas"],
            eps=s["eps"], weight_decay=s["weight_decay"], state_bits=case["bits"], seed=s["seed"],
            state={"step": s["step"], "exp_avg": s["m"], "exp_avg_sq": s["v"], "exp_avg_scale": s["m_scale"],
                   "exp_avg_sq_scale": s["v_scale"]})
    return s


def _prepare_policy(case, g):
    lengths = torch.tensor(_lengths(case), device=DEV)
    T, B = int(lengths.sum()), case["sequences"]
    cu = torch.zeros(B + 1, dtype=torch.int64, device=DEV)
    cu[1:] = lengths.cumsum(0)
    logp = -torch.empty(T, device=DEV).exponential_(1.0, generator=g)
    s = {"case": case, "cu_seqlens": cu, "T": T, "clip_low": 0.2, "clip_high": 0.28,
         "kl_coef": 0.05 if case["ref"] else 0.0, "entropy_coef": 0.01 if case["entropy"] else 0.0}
    s["old_logp"] = logp + 0.15 * torch.randn(T, generator=g, device=DEV)
    s["ref_logp"] = logp + 0.3 * torch.randn(T, generator=g, device=DEV) if case["ref"] else None
    s["entropy"] = torch.rand(T, generator=g, device=DEV) * 3 if case["entropy"] else None
    s["advantages"] = torch.randn(B if case["per_sequence"] else T, generator=g, device=DEV) + 0.2
    s["mask"] = None
    if case["masked"]:
        # a prompt at the start of each sequence, its rows' log-probabilities NaN; one sequence in eight has no answer
        place = torch.arange(T, device=DEV) - torch.repeat_interleave(cu[:-1], lengths, output_size=T)
        share = torch.clamp_max(torch.rand(B, generator=g, device=DEV) * 2 * case["masked"], 0.97)
        none = (torch.rand(B, generator=g, device=DEV) < 0.125) & (torch.arange(B, device=DEV) > 0)
        share = torch.where(none, torch.ones_like(share), share)
        prompt = torch.repeat_interleave((share * lengths).long(), lengths, output_size=T)
        s["mask"] = place >= prompt
        logp = torch.where(s["mask"], logp, torch.full_like(logp, math.nan))
    s["logp"] = logp
    return s


# ------------------------------------------------------------------------ one pass

def run(state):
    op = state["case"]["op"]
    if op == "norm":
        backward = state["case"]["direction"] == "backward"
        if own:
            return _own_norm_backward(state) if backward else _own_norm(state)
        return _plain_norm_backward(state) if backward else _plain_norm(state)
    if op == "adamw":
        return _own_adamw(state) if own else _plain_adamw(state)
    return _own_policy(state) if own else _plain_policy(state)


def _own_norm(s):
    from invariant_token_logprobs_gb300 import train
    return tuple(train.residual_norm(s["residual"], s["branch"], weight=s["weight"], branch_weight=s["branch_weight"],
                                     gate=s["gate"], residual_scale=s["residual_scale"],
                                     branch_scale=s["branch_scale"], eps=s["eps"]))


def _own_norm_backward(s):
    from invariant_token_logprobs_gb300 import train
    return tuple(train.residual_norm_backward(
        s["grad_normed"], s["grad_residual"], s["residual"], s["rstd"], branch=s["branch"], weight=s["weight"],
        branch_weight=s["branch_weight"], branch_rstd=s["branch_rstd"], gate=s["gate"],
        residual_scale=s["residual_scale"], branch_scale=s["branch_scale"]))


def _own_adamw(s):
    optimizer = s["optimizer"]
    norm = optimizer.step(max_norm=s["max_norm"])
    m, v = optimizer.state_values()
    return s["param"], s["copy"], m, v, norm


def _own_policy(s):
    from invariant_token_logprobs_gb300 import train
    case = s["case"]
    return tuple(train.policy_loss(s["logp"], s["old_logp"], s["advantages"], mask=s["mask"], ref_logp=s["ref_logp"],
                                   entropy=s["entropy"], cu_seqlens=s["cu_seqlens"], reduction=case["reduction"],
                                   per_sequence=case["per_sequence"], clip_low=s["clip_low"], clip_high=s["clip_high"],
                                   kl_coef=s["kl_coef"], entropy_coef=s["entropy_coef"]))


# ------------------------------------------------------------------------ plain forms

def _norm_stream(s):
    """The new residual stream in float32 and the reciprocal roots of both norms."""
    n, branch_rstd = s["branch"].float(), None
    if s["branch_weight"] is not None:
        branch_rstd = torch.rsqrt((n * n).mean(1) + s["eps"])
        n = n * branch_rstd[:, None] * s["branch_weight"].float()
    if s["gate"] is not None:
        n = n * s["gate"].float()
    new = s["residual_scale"] * s["residual"].float() + s["branch_scale"] * n
    return new, torch.rsqrt((new * new).mean(1) + s["eps"]), branch_rstd


def _plain_norm(s):
    new, rstd, branch_rstd = _norm_stream(s)
    normed = new * rstd[:, None] * s["weight"].float()
    return normed.to(s["branch"].dtype), new.to(s["residual"].dtype), rstd, branch_rstd


def _plain_norm_backward(s):
    dh, x = s["grad_normed"].float(), s["residual"].float() * s["rstd"][:, None]
    grad_weight = (dh * x).sum(0)
    dx = dh * s["weight"].float()
    D = s["grad_residual"].float() + s["rstd"][:, None] * (dx - x * (dx * x).mean(1, keepdim=True))
    grad_residual = (s["residual_scale"] * D).to(s["residual"].dtype)
    y = s["branch"].float()
    hat = y * s["branch_rstd"][:, None] if s["branch_weight"] is not None else y
    n = hat * s["branch_weight"].float() if s["branch_weight"] is not None else y
    dn = s["branch_scale"] * D
    grad_gate = grad_branch_weight = None
    if s["gate"] is not None:
        grad_gate = dn * n
        grad_gate = grad_gate.to(s["gate"].dtype) if s["gate"].dim() == 2 else grad_gate.sum(0)
        dn = dn * s["gate"].float()
    if s["branch_weight"] is not None:
        grad_branch_weight = (dn * hat).sum(0)
        dn = dn * s["branch_weight"].float()
        dn = s["branch_rstd"][:, None] * (dn - hat * (dn * hat).mean(1, keepdim=True))
    return grad_residual, dn.to(s["branch"].dtype), grad_weight, grad_branch_weight, grad_gate


def _random_words(groups, step, seed):
    """Four 32-bit words for each group of four elements: Philox 4x32 with 7 rounds
    (Salmon et al., SC11) at counter (group, step) and key seed."""
    low = 0xFFFFFFFF
    group = torch.arange(groups, dtype=torch.int64, device=DEV)
    c = [group & low, group >> 32, torch.full_like(group, step & low), torch.full_like(group, step >> 32)]
    k0, k1 = seed & low, (seed >> 32) & low

    def one(c, k0, k1):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        return [((b >> 32) & low) ^ c[1] ^ k0, b & low, ((a >> 32) & low) ^ c[3] ^ k1, a & low]

    c = one(c, k0, k1)
    c = one(c, (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low)
    c = one(c, (k0 + 2 * 0x9E3779B9) & low, (k1 + 2 * 0xBB67AE85) & low)
    c = one(c, (k0 + 3 * 0x9E3779B9) & low, (k1 + 3 * 0xBB67AE85) & low)
    c = one(c, (k0 + 4 * 0x9E3779B9) & low, (k1 + 4 * 0xBB67AE85) & low)
    c = one(c, (k0 + 5 * 0x9E3779B9) & low, (k1 + 5 * 0xBB67AE85) & low)
    c = one(c, (k0 + 6 * 0x9E3779B9) & low, (k1 + 6 * 0xBB67AE85) & low)
    return torch.stack(c, 1).view(-1)


# An 8-bit moment is a magnitude code and a scale, the block's largest magnitude. Code c > 0 is
# the float with the bits (c + first) << shift: 1 at the top code, 2^-16 at the lowest, each
# octave in 8 steps (the first moment, 7 bits and a sign) or 16 (the root of the second moment,
# 8 bits). Code 0 is zero. Rounding goes up with the probability of the part that is cut off.

def _code(signed):
    return (20, 889, 1.25 * 2.0 ** -36) if signed else (19, 1777, 1.125 * 2.0 ** -35)


def _encode(x, signed, words):
    shift, first, low = _code(signed)
    x = x.view(-1, BLOCK)
    scale = x.abs().amax(1)
    scale = torch.where(scale < 2.0 ** -100, torch.zeros_like(scale), scale)
    inverse = torch.where(scale > 0, 1.0 / scale, scale)
    part = torch.clamp_max(x.abs() * inverse[:, None], 1.0).view(-1)
    r = (((words & 0xFFFF) if signed else (words >> 16) & 0xFFFF) << (shift - 16)).to(torch.int32)
    c = ((part.view(torch.int32) + r) >> shift) - first
    c = torch.where(part.view(torch.int32) < ((first + 1) << shift), (part > r.float() * low).to(torch.int32), c)
    if signed:
        c = torch.where((x.view(-1) < 0) & (c > 0), c + 128, c)
    return c.to(torch.uint8), scale


def _decode(code, scale, signed):
    shift, first, _ = _code(signed)
    c = code.to(torch.int32)
    mag = (c & 127) if signed else c
    value = torch.where(mag > 0, (mag + first) << shift, torch.zeros_like(mag)).view(torch.float32)
    if signed:
        value = torch.where(c >= 128, -value, value)
    return (value.view(-1, BLOCK) * scale[:, None]).view(-1)


def _plain_adamw(s):
    bits8 = s["case"]["bits"] == 8
    b1, b2 = s["betas"]
    s["step"] += 1
    g, norm = s["grad"].float(), None
    if s["max_norm"] is not None:
        norm = torch.sqrt((g * g).sum())
        g = g * torch.clamp_max(s["max_norm"] / (norm + 1e-6), 1.0)
    m = _decode(s["m"], s["m_scale"], True) if bits8 else s["m"]
    v = s["v"]
    if bits8:
        v = _decode(s["v"], s["v_scale"], False)
        v = v * v
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * (g * g)
    root = torch.sqrt(v)
    change = m / (root * (1 / math.sqrt(1 - b2 ** s["step"])) + s["eps"])
    kept = (s["param"].view(-1, ALIGN) * (1 - s["lr"] * s["decay_rows"])).view(-1)
    s["param"] = kept - (s["lr"] / (1 - b1 ** s["step"])) * change
    copy = s["param"].to(torch.bfloat16) if s["copy"] is not None else None
    if not bits8:
        s["m"], s["v"] = m, v
        return s["param"], copy, m, v, norm
    words = _random_words(m.numel() // 4, s["step"], s["seed"])
    s["m"], s["m_scale"] = _encode(m, True, words)
    s["v"], s["v_scale"] = _encode(root, False, words)
    root = _decode(s["v"], s["v_scale"], False)
    return s["param"], copy, _decode(s["m"], s["m_scale"], True), root * root, norm


def _plain_policy(s):
    case, T, cu = s["case"], s["T"], s["cu_seqlens"]
    sequence = torch.repeat_interleave(torch.arange(case["sequences"], device=DEV), cu[1:] - cu[:-1], output_size=T)
    zero = torch.zeros((), device=DEV)
    keep = s["mask"] if s["mask"] is not None else torch.ones(T, dtype=torch.bool, device=DEV)
    A = s["advantages"][sequence] if case["per_sequence"] else s["advantages"]
    if case["reduction"] == "token":
        w = torch.where(keep, 1.0 / keep.float().sum().clamp_min(1.0), zero)
    else:
        n = torch.zeros(case["sequences"], device=DEV).index_add_(0, sequence, keep.float())
        w = torch.where(keep, (1.0 / (n.clamp_min(1.0) * (n > 0).float().sum().clamp_min(1.0)))[sequence], zero)
    delta = torch.where(keep, s["logp"] - s["old_logp"], zero)
    high, low = math.log1p(s["clip_high"]), math.log1p(-s["clip_low"])
    over, under = (A > 0) & (delta > high), (A < 0) & (delta < low)
    clipped = over | under
    ratio = torch.exp(delta)
    bounded = torch.where(over, 1 + s["clip_high"], torch.where(under, 1 - s["clip_low"], ratio))
    policy = (w * torch.where(keep, -A * bounded, zero)).sum()
    grad = torch.where(keep & ~clipped, -A * ratio, zero)
    kl = entropy = zero
    if s["ref_logp"] is not None:
        r = torch.where(keep, s["ref_logp"] - s["logp"], zero)
        up = torch.expm1(r)
        kl = (w * (up - r)).sum()
        grad = grad - s["kl_coef"] * up
    grad_entropy = None
    if s["entropy"] is not None:
        entropy = (w * torch.where(keep, s["entropy"], zero)).sum()
        grad_entropy = -s["entropy_coef"] * w
    loss = policy + s["kl_coef"] * kl - s["entropy_coef"] * entropy
    share = (w * (clipped & keep).float()).sum()
    return torch.stack([loss, policy, kl, entropy, share]), w * grad, grad_entropy


# ------------------------------------------------------------------------ work

def work(case):
    if case["op"] == "norm":
        T, d, r, a, w = case["T"], case["d"], BYTES[case["residual"]], BYTES[case["act"]], BYTES[case["weight"]]
        vectors = d * w * (1 + case["post"]) + (d * a if case["gate"] == "channel" else 0)
        rows = T * d * a if case["gate"] == "token" else 0
        if case["direction"] == "forward":
            # the stream and the block's output in, the new stream and its norm out
            return {"bytes": T * d * 2 * (r + a) + rows + vectors + 4 * T * (1 + case["post"]), "flops": 10 * T * d}
        # the stream, the block's output and both gradients in, two gradients out
        grads = 4 * d * (1 + case["post"] + (case["gate"] == "channel"))
        return {"bytes": T * d * 3 * (r + a) + 2 * rows + vectors + grads + 4 * T * (1 + case["post"]), "flops": 30 * T * d}
    if case["op"] == "adamw":
        n = sum(_sizes(case))
        state = 16 if case["bits"] == 32 else 4 + 16 / BLOCK
        # 8-bit moments are returned as the values they stand for
        values = 8 if case["bits"] == 8 else 0
        return {"bytes": n * (8 + BYTES[case["grad"]] + state + values + (2 if case["copy"] else 0)), "flops": 20 * n}
    T = sum(_lengths(case))
    each = 8 + (0 if case["per_sequence"] else 4) + (4 if case["ref"] else 0) + (4 if case["entropy"] else 0)
    each += (1 if case["masked"] else 0) + 4 + (4 if case["entropy"] else 0)
    rows = 8 * (case["sequences"] + 1) + (4 * case["sequences"] if case["per_sequence"] else 0)
    return {"bytes": T * each + rows, "flops": 25 * T}


# ------------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "adamw": _exact_adamw, "policy": _exact_policy}[case["op"]](s)


def _exact_norm(s):
    d = s["case"]["d"]
    post, gate = s["branch_weight"], s["gate"]
    y, w = s["branch"].double(), s["weight"].double()
    wb = 1.0 if post is None else post.double()
    k = s["branch_scale"] * (1.0 if gate is None else gate.double())
    if s["case"]["direction"] == "forward":
        ry = 1.0 if post is None else (y.square().sum(1, keepdim=True) / d + s["eps"]).pow(-0.5)
        new = s["residual"].double() * s["residual_scale"] + k * (y * ry * wb)
        rn = (new.square().sum(1, keepdim=True) / d + s["eps"]).pow(-0.5)
        return new * rn * w, new, rn[:, 0], None if post is None else ry[:, 0]
    # dL/d(new) = dnew + J^T dh for h = new * rn(new) * w, and the same for the branch's norm
    rn, ry = s["rstd"].double()[:, None], 1.0 if post is None else s["branch_rstd"].double()[:, None]
    new, dh = s["residual"].double(), s["grad_normed"].double()
    dot = (dh * w * new).sum(1, keepdim=True)
    D = s["grad_residual"].double() + rn * w * dh - new * dot * rn ** 3 / d
    dk = D * (y * ry * wb)
    e = D * k * wb
    dy = e * ry
    if post is not None:
        dy = dy - y * (e * y).sum(1, keepdim=True) * ry ** 3 / d
    gw = (dh * new * rn).sum(0)
    gb = None if post is None else (D * k * y * ry).sum(0)
    gg = None if gate is None else s["branch_scale"] * (dk if gate.dim() == 2 else dk.sum(0))
    return D * s["residual_scale"], dy, gw, gb, gg


def _exact_round(x, signed, words):
    """The 8-bit values of x (float64) under the same random words."""
    steps = 8.0 if signed else 16.0
    blocks = x.view(-1, BLOCK)
    top = blocks.abs().amax(1, keepdim=True)
    top = torch.where(top < 2.0 ** -100, torch.zeros_like(top), top)
    part = torch.where(top > 0, blocks.abs() / top, torch.zeros_like(blocks))
    u = (((words if signed else words >> 16) & 0xFFFF).double() / 65536).view_as(part)
    lowest = 1.25 * 2.0 ** -16 if signed else 1.125 * 2.0 ** -16
    mantissa, exponent = torch.frexp(part)
    octave = torch.ldexp(torch.ones_like(part), exponent - 1)
    near = octave * (1 + torch.floor((2 * mantissa - 1) * steps + u) / steps)
    near = torch.where(part < lowest, lowest * (part > u * lowest).double(), near)
    return (torch.sign(blocks) * near * top).view(-1)


def _exact_adamw(s):
    bits8 = s["case"]["bits"] == 8
    b1, b2 = s["betas"]
    t = s["step"] + 1
    g, norm = s["grad"].double(), None
    if s["max_norm"] is not None:
        norm = g.square().sum().sqrt()
        g = g * min(1.0, s["max_norm"] / (float(norm) + 1e-6))
    m0 = _decode(s["m"], s["m_scale"], True).double() if bits8 else s["m"].double()
    v0 = _decode(s["v"], s["v_scale"], False).double().square() if bits8 else s["v"].double()
    m = m0 + (1 - b1) * (g - m0)
    v = v0 + (1 - b2) * (g.square() - v0)
    del m0, v0, g
    wd = torch.zeros(s["at"][-1] // ALIGN, 1, dtype=torch.float64, device=DEV)
    for a, b, d in zip(s["at"][:-1], s["at"][1:], s["weight_decay"]):
        wd[a // ALIGN:b // ALIGN] = d
    p = (s["param"].double().view(-1, ALIGN) * (1 - s["lr"] * wd)).view(-1)
    p -= s["lr"] * (m / (1 - b1 ** t)) / ((v / (1 - b2 ** t)).sqrt() + s["eps"])
    copy = p if s["copy"] is not None else None
    if bits8:
        words = _random_words(m.numel() // 4, t, s["seed"])
        m, v = _exact_round(m, True, words), _exact_round(v.sqrt(), False, words).square()
    return p, copy, m, v, norm


def _exact_policy(s):
    case, T, cu = s["case"], s["T"], s["cu_seqlens"]
    sequence = torch.searchsorted(cu[1:], torch.arange(T, device=DEV), right=True)
    keep = s["mask"] if s["mask"] is not None else torch.ones(T, dtype=torch.bool, device=DEV)
    at = keep.nonzero()[:, 0]
    seq = sequence[at]
    A = (s["advantages"][seq] if case["per_sequence"] else s["advantages"][at]).double()
    if case["reduction"] == "token":
        w = torch.full((at.numel(),), 1.0 / max(1, at.numel()), dtype=torch.float64, device=DEV)
    else:
        n = torch.bincount(seq, minlength=case["sequences"])
        w = 1.0 / (n[seq].double() * max(1, int((n > 0).sum())))
    logp, old = s["logp"][at], s["old_logp"][at]
    # the clip is decided on the float32 difference and the limits rounded to float32
    delta = logp - old
    over = (A > 0) & (delta > torch.tensor(math.log1p(s["clip_high"]), dtype=torch.float32, device=DEV))
    under = (A < 0) & (delta < torch.tensor(math.log1p(-s["clip_low"]), dtype=torch.float32, device=DEV))
    ratio = (logp.double() - old.double()).exp()
    surrogate = -A * torch.where(over, 1 + s["clip_high"], torch.where(under, 1 - s["clip_low"], ratio))
    grad = torch.where(over | under, torch.zeros_like(A), -A * ratio)
    kl = entropy = 0.0
    if s["ref_logp"] is not None:
        r = s["ref_logp"][at].double() - logp.double()
        kl = float((w * (r.expm1() - r)).sum())
        grad = grad - s["kl_coef"] * r.expm1()
    full = torch.zeros(T, dtype=torch.float64, device=DEV)
    grad_entropy = None
    if s["entropy"] is not None:
        entropy = float((w * s["entropy"][at].double()).sum())
        grad_entropy = full.index_copy(0, at, -s["entropy_coef"] * w)
    policy = float((w * surrogate).sum())
    stats = [policy + s["kl_coef"] * kl - s["entropy_coef"] * entropy, policy, kl, entropy,
             float((w * (over | under).double()).sum())]
    return torch.tensor(stats, dtype=torch.float64), full.index_copy(0, at, w * grad), grad_entropy
