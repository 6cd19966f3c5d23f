"""The operators of learning through a packed head, as a training program calls them, with their plain forms.

Three operators follow one another in a step of policy or preference training on top of a frozen packed head
(`lse_argmax` gives the per-token cross-entropy `ce = -log p(token)` that they start from):

policy loss       ce, ce_old, advantages (and ce_ref) -> loss, d loss / d ce, three statistics
preference loss   ce (and ce_ref) of chosen and rejected sequences -> loss, d loss / d ce, rewards
head gradient     d loss / d ce -> d loss / d hidden, through the softmax over the whole vocabulary and the packed rows

Plain forms: elementary torch operations, in 32 bits for the head. The losses are in 64: log-ratios lie next to a
clipping border or near zero, and a loss of normalised advantages is the small sum of large terms of both signs.
"""
import math

import torch

own = False

SCALE_STD = {"s_L": 2e-3, "s_R": 1e-3, "s_res": 3e-3, "s_A": 2e-3, "s_B": 2.5e-4}


# ------------------------------------------------------------------ the cases
def _grad(name, V, d, r_c, r_r, g, g_B, T):
    return {"name": name, "op": "grad", "V": V, "d": d, "r_c": r_c, "r_r": r_r, "g": g, "g_B": g_B, "T": T}


def _policy(name, S, mean, ref, masked, per, reduction):
    return {"name": name, "op": "policy", "S": S, "mean": mean, "ref": ref, "masked": masked, "per": per,
            "reduction": reduction}


def _preference(name, N, mean, ref, masked, kind, average):
    return {"name": name, "op": "preference", "N": N, "mean": mean, "ref": ref, "masked": masked, "kind": kind,
            "average": average}


def listed():
    return [
        # The head built from a dense one in the tests: a few tokens, where launches are the cost.
        _grad("grad tiny head 4 tokens", 1024, 256, 32, 8, 64, 64, 4),
        # One token through a head of odd size: an online update after each sampled token.
        _grad("grad odd head 1 token", 32003, 2048, 256, 32, 32, 64, 1),
        # The two head shapes of the benchmark at their decode batches: short rollouts, a step per batch.
        _grad("grad 262144 x 2560 16 tokens", 262144, 2560, 384, 64, 128, 128, 16),
        _grad("grad 151936 x 4096 64 tokens", 151936, 4096, 512, 64, 128, 128, 64),
        # A plain INT4 head (no low-rank branches) and a ragged packed batch of sequences.
        _grad("grad INT4 head 777 tokens", 65531, 1024, 0, 0, 16, 128, 777),
        # A training micro-batch at the prefill size of the benchmark.
        _grad("grad 151936 x 4096 4096 tokens", 151936, 4096, 512, 64, 128, 128, 4096),
        # A handful of short rollouts.
        _policy("policy 3 short rollouts", 3, 100, False, False, "token", "tokens"),
        # One prompt group of 64 rollouts of some thousand tokens, prompts masked, with a reference model.
        _policy("policy 64 rollouts", 64, 1024, True, True, "sequence", "tokens"),
        # A whole step's rollouts at once, sequence by sequence.
        _policy("policy 512 rollouts", 512, 2048, True, True, "sequence", "sequences"),
        # Two pairs of short answers; a batch of pairs; a few pairs of very long answers.
        _preference("preference 2 pairs", 2, 120, True, True, "sigmoid", False),
        _preference("preference 256 pairs", 256, 500, True, True, "sigmoid", False),
        _preference("preference 8 long pairs", 8, 24000, True, False, "squared", True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["grad", "grad", "policy", "preference"])
    if op == "policy":
        S = _log(rng, 1, 1024)
        c = _policy("", S, max(1, min(_log(rng, 1, 8192), (1 << 20) // S)), rng.random() < 0.5, rng.random() < 0.5,
                    rng.choice(["token", "sequence"]), rng.choice(["tokens", "sequences", "sum"]))
    elif op == "preference":
        N = _log(rng, 1, 1024)
        c = _preference("", N, max(1, min(_log(rng, 1, 32768), (1 << 18) // N)), rng.random() < 0.7, rng.random() < 0.5,
                        rng.choice(["sigmoid", "hinge", "squared"]), rng.random() < 0.3)
    else:
        d = 128 * rng.randint(2, 32)
        V = _log(rng, 1000, 160000)
        most = 4096 * 151936 * 4096 // (V * d)
        c = _grad("", V, d, rng.choice([0, 100, 256, 512]), rng.choice([0, 8, 64]), rng.choice([16, 32, 64, 128]),
                  rng.choice([32, 64, 128]), max(1, min(_log(rng, 1, 4096), most)))
    del c["name"]
    return c


# ----------------------------------------------------------------- the inputs
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) + 20260802)


def _components(case, gen):
    """Packed components on the device: codes as int8, scales as fp16 (half-normal, as in the tests' heads)."""
    V, d, r_c, r_r = case["V"], case["d"], case["r_c"], case["r_r"]

    def codes(lo, hi, *shape):
        return torch.randint(lo, hi + 1, shape, generator=gen, device="cuda", dtype=torch.int8)

    def scales(name, *shape):
        return (torch.randn(shape, generator=gen, device="cuda").abs() * SCALE_STD[name]).half()

    return {"L": codes(-16, 15, V, r_c), "s_L": scales("s_L", V), "R": codes(-128, 127, r_c, d), "s_R": scales("s_R", r_c),
            "q": codes(-8, 7, V, d), "s_res": scales("s_res", V, d // case["g"]),
            "A": codes(-128, 127, V, r_r), "s_A": scales("s_A", V),
            "B": codes(-128, 127, r_r, d), "s_B": scales("s_B", r_r, d // case["g_B"])}


def _grad_inputs(case, seed):
    """A head, anisotropic hidden states whose logits have a spread of about 2.5, tokens sampled from the head's own
    softmax, its log-sum-exp, and the loss's gradients: a third of the tokens (prompts) have none."""
    gen = _generator(seed)
    c = _components(case, gen)
    V, d, T = case["V"], case["d"], case["T"]
    lam = torch.arange(1, d + 1, device="cuda", dtype=torch.float32) ** -0.75
    h = (torch.randn(T, d, generator=gen, device="cuda") * lam) @ torch.randn(d, d, generator=gen, device="cuda")
    w = _dense(c, torch.float32)
    y = h @ w.T
    h = (h * (2.5 / y.std())).bfloat16()
    y = h.float() @ w.T
    lse = torch.logsumexp(y.double(), 1).float()
    u = torch.rand(T, V, generator=gen, device="cuda").clamp_(1e-7, 1 - 1e-7)
    targets = (y - torch.log(-torch.log(u))).argmax(1).int()
    del y, u, w
    g = torch.randn(T, generator=gen, device="cuda") / T
    if T > 2:
        g = torch.where(torch.rand(T, generator=gen, device="cuda") < 1 / 3, torch.zeros_like(g), g)
    return c, h, targets, lse, g


def _lengths(n, mean, gen):
    """Running sums of n lengths, about half to one and a half times the mean, n * mean tokens in all."""
    run = (torch.rand(n, generator=gen, device="cuda") + 0.5).double().cumsum(0)
    cu = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    cu[1:] = (run / run[-1] * (n * mean)).round()
    return cu


def _token_inputs(case, seed):
    """Cross-entropies of sampled tokens (mostly small, some of several nats), those of the policy that sampled them and
    of a reference model, advantages, and a mask without the prompts (the first part of a sequence) if there is one."""
    gen = _generator(seed)
    n = case["S"] if case["op"] == "policy" else 2 * case["N"]
    cu = _lengths(n, case["mean"], gen)
    T = int(cu[-1])

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    ce = normal(T).exp() * 0.5
    spread = 0.15 if case["op"] == "policy" else 0.05
    s = {"cu": cu, "ce": ce, "ref": (ce + spread * normal(T)).clamp_(min=0) if case["ref"] else None}
    if case["op"] == "policy":
        s["old"] = (ce + 0.15 * normal(T)).clamp_(min=0)
        s["adv"] = normal(T if case["per"] == "token" else n)
    s["mask"] = None
    if case["masked"]:
        at = torch.arange(T, device="cuda")
        seq = torch.searchsorted(cu[1:].long(), at, right=True)
        start, length = cu[seq].long(), (cu[seq + 1] - cu[seq]).long()
        prompt = torch.rand(n, generator=gen, device="cuda")[seq] * 0.6 * length
        s["mask"] = (at - start) >= prompt.long()
    return s


def prepare(case, seed):
    if case["op"] != "grad":
        return {"case": case, **_token_inputs(case, seed)}
    c, h, targets, lse, g = _grad_inputs(case, seed)
    s = {"case": case, "h": h, "targets": targets, "lse": lse, "g": g}
    if own:
        import numpy as np

        import quantized_output_head_b200 as qoh
        host = {k: v.cpu().numpy() for k, v in c.items()}
        host = {k: v.view(np.uint16) if v.dtype == np.float16 else v for k, v in host.items()}
        s["head"] = qoh.PackedHead(case["V"], case["d"], case["r_c"], case["r_r"], case["g"], case["g_B"], host)
    else:
        s["c"] = c
    return s


# ------------------------------------------------------------ the plain forms
def _dense(c, dtype):
    """The rows that the packed components stand for: core, residual with its group scales, correction."""
    def groups(codes, scales):
        return (codes.to(dtype).view(codes.shape[0], scales.shape[1], -1) * scales.to(dtype)[:, :, None]).view(codes.shape)

    w = groups(c["q"], c["s_res"])
    if c["R"].shape[0]:
        w = w + (c["L"].to(dtype) * c["s_L"].to(dtype)[:, None]) @ (c["R"].to(dtype) * c["s_R"].to(dtype)[:, None])
    if c["B"].shape[0]:
        w = w + (c["A"].to(dtype) * c["s_A"].to(dtype)[:, None]) @ groups(c["B"], c["s_B"])
    return w


def _grad_plain(s):
    w = _dense(s["c"], torch.float32)
    p = torch.exp(s["h"].float() @ w.T - s["lse"][:, None])
    p[torch.arange(p.shape[0], device="cuda"), s["targets"].long()] -= 1
    return ((p * s["g"][:, None]) @ w).bfloat16()


def _sequence_of(cu, T):
    return torch.searchsorted(cu[1:].long(), torch.arange(T, device="cuda"), right=True)


def _sums(x, cu):
    """Sums over each sequence, in 64 bits."""
    run = torch.cat([x.new_zeros(1, dtype=torch.float64), x.double().cumsum(0)])
    return run[cu[1:].long()] - run[cu[:-1].long()]


CLIP_LOW, CLIP_HIGH, KL_COEF, BETA = 0.2, 0.28, 0.04, 0.1


def _policy_plain(s):
    case, ce, cu = s["case"], s["ce"], s["cu"]
    T = ce.numel()
    seq = _sequence_of(cu, T)
    keep = torch.ones_like(ce, dtype=torch.bool) if s["mask"] is None else s["mask"]
    adv = (s["adv"] if case["per"] == "token" else s["adv"][seq]).double()
    delta = s["old"].double() - ce.double()
    ratio = delta.exp()
    cut = torch.where(adv > 0, delta > math.log1p(CLIP_HIGH), (adv < 0) & (delta < math.log1p(-CLIP_LOW)))
    clipped = 1 - CLIP_LOW + (CLIP_HIGH + CLIP_LOW) * (adv > 0).double()
    loss = -adv * torch.where(cut, clipped, ratio)
    grad = torch.where(cut, torch.zeros_like(ratio), adv * ratio)
    kl_old = torch.expm1(delta) - delta
    kl_ref = torch.zeros_like(delta)
    if s["ref"] is not None:
        delta = ce.double() - s["ref"].double()
        kl_ref = torch.expm1(delta) - delta
        loss = loss + KL_COEF * kl_ref
        grad = grad + KL_COEF * torch.expm1(delta)
    count = _sums(keep, cu)
    total = keep.sum()
    if case["reduction"] == "tokens":
        weight = (keep / total.clamp(min=1)).double()
    elif case["reduction"] == "sequences":
        weight = keep / (count.clamp(min=1) * (count > 0).sum().clamp(min=1))[seq]
    else:
        weight = keep.double()
    stats = torch.stack([(keep & cut).sum().double(), (keep * kl_old).sum(), (keep * kl_ref).sum()])
    return (loss * weight).sum().float(), (grad * weight).float(), (stats / total.clamp(min=1)).float()


def _preference_plain(s):
    case, ce, cu, N = s["case"], s["ce"], s["cu"], s["case"]["N"]
    seq = _sequence_of(cu, ce.numel())
    keep = torch.ones_like(ce, dtype=torch.bool) if s["mask"] is None else s["mask"]
    x = -ce.double() if s["ref"] is None else s["ref"].double() - ce.double()
    each = torch.ones(2 * N, device="cuda", dtype=torch.float64)
    if case["average"]:
        each = 1 / _sums(keep, cu).clamp(min=1)
    score = _sums(x * keep, cu) * each
    gap = score[:N] - score[N:]
    if case["kind"] == "sigmoid":
        m = BETA * gap
        loss, slope = torch.log1p(torch.exp(-m.abs())) + (-m).clamp(min=0), -BETA / (1 + torch.exp(m))
    elif case["kind"] == "hinge":
        loss, slope = (1 - BETA * gap).clamp(min=0), -BETA * (BETA * gap < 1).double()
    else:
        loss, slope = (gap - 0.5 / BETA) ** 2, 2 * (gap - 0.5 / BETA)
    to = torch.cat([-slope, slope]) * each / N
    return loss.mean().float(), torch.where(keep, to[seq], 0.0).float(), (BETA * score).view(2, N).float()


def run(s):
    case = s["case"]
    if own:
        import quantized_output_head_b200 as qoh
        if case["op"] == "grad":
            return s["head"].grad_hidden(s["h"], s["targets"], s["lse"], s["g"])
        if case["op"] == "policy":
            return qoh.policy_loss(s["ce"], s["old"], s["adv"], s["cu"], mask=s["mask"], ce_ref=s["ref"],
                                   clip_low=CLIP_LOW, clip_high=CLIP_HIGH, kl_coef=KL_COEF,
                                   advantage_per=case["per"], reduction=case["reduction"])
        return qoh.preference_loss(s["ce"], s["cu"], mask=s["mask"], ce_ref=s["ref"], beta=BETA, kind=case["kind"],
                                   average=case["average"])
    if case["op"] == "grad":
        return _grad_plain(s)
    return _policy_plain(s) if case["op"] == "policy" else _preference_plain(s)


# ---------------------------------------------------------------- their work
def work(case):
    if case["op"] == "grad":
        V, d, r_c, r_r, T = case["V"], case["d"], case["r_c"], case["r_r"], case["T"]
        head = V * (5 * r_c / 8 + 2 + d / 2 + 2 * d / case["g"] + r_r + 2) + r_c * (d + 2) + r_r * (d + 2 * d / case["g_B"])
        # hidden states in and their gradients out (2 bytes), targets, log-sum-exp, gradients in (4 bytes)
        return {"bytes": head + T * (4 * d + 12), "flops": 2 * (2 * T * V * (d + r_c + r_r) + 2 * T * d * (r_c + r_r))}
    policy = case["op"] == "policy"
    n = case["S"] if policy else 2 * case["N"]
    T = n * case["mean"]
    each = 4 + 4 + (4 if case["ref"] else 0) + (1 if case["masked"] else 0)
    if policy:
        each += 4 + (4 if case["per"] == "token" else 0)
    return {"bytes": T * each + 12 * n, "flops": T * (20 if policy else 4)}


# ------------------------------------------------------ the values in 64 bits
def exact(case, seed):
    if case["op"] == "grad":
        return _exact_grad(case, seed)
    s = _token_inputs(case, seed)
    ce = s["ce"].double()
    cu = s["cu"].cpu().tolist()
    keep = torch.ones_like(ce) if s["mask"] is None else s["mask"].double()
    spans = list(zip(cu[:-1], cu[1:]))
    owner = torch.repeat_interleave(torch.arange(len(spans), device="cuda"), torch.tensor([b - a for a, b in spans], device="cuda"))
    counts = torch.zeros(len(spans), dtype=torch.float64, device="cuda").index_add_(0, owner, keep)
    if case["op"] == "preference":
        N = case["N"]
        logratio = keep * ((s["ref"].double() if s["ref"] is not None else 0.0) - ce)
        score = torch.zeros_like(counts).index_add_(0, owner, logratio).requires_grad_(True)
        mean = score / counts.clamp(min=1) if case["average"] else score
        gap = mean[:N] - mean[N:]
        if case["kind"] == "sigmoid":
            losses = -torch.nn.functional.logsigmoid(BETA * gap)
        elif case["kind"] == "hinge":
            losses = torch.relu(1 - BETA * gap)
        else:
            losses = (gap - 1 / (2 * BETA)).square()
        loss = losses.mean()
        loss.backward()
        return loss.detach(), -score.grad[owner] * keep, BETA * mean.detach().view(2, N)
    x = ce.clone().requires_grad_(True)
    adv = s["adv"].double() if case["per"] == "token" else s["adv"].double()[owner]
    ratio = torch.exp(s["old"].double() - x)
    inside = ratio.clamp(1 - CLIP_LOW, 1 + CLIP_HIGH)
    terms = torch.maximum(-adv * ratio, -adv * inside)
    kl_old = (ratio - 1) - torch.log(ratio)
    kl_ref = torch.zeros_like(x)
    if s["ref"] is not None:
        kl_ref = torch.expm1(x - s["ref"].double()) - (x - s["ref"].double())
    terms = terms + KL_COEF * kl_ref
    total = max(1.0, float(keep.sum()))
    if case["reduction"] == "tokens":
        loss = (terms * keep).sum() / total
    elif case["reduction"] == "sequences":
        means = torch.zeros_like(counts).index_add(0, owner, terms * keep) / counts.clamp(min=1)
        loss = means.sum() / max(1.0, float((counts > 0).sum()))
    else:
        loss = (terms * keep).sum()
    loss.backward()
    bound = ((adv * ratio) > (adv * inside)).double()   # the clipped value is the smaller one
    stats = torch.stack([(bound * keep).sum(), (kl_old * keep).sum(), (kl_ref * keep).sum()]).detach() / total
    return loss.detach(), x.grad, stats


def _exact_grad(case, seed):
    """Rows of the vocabulary in blocks: each adds its softmax-weighted rows, the token's own row is taken off."""
    c, h, targets, lse, g = _grad_inputs(case, seed)
    h, lse, g, targets = h.double(), lse.double(), g.double(), targets.long()
    right_core = c["R"].double() * c["s_R"].double()[:, None]
    right_corr = c["B"].double() * c["s_B"].double().repeat_interleave(case["g_B"], 1)
    out = torch.zeros_like(h)
    for a in range(0, case["V"], 32768):
        b = min(case["V"], a + 32768)
        rows = c["q"][a:b].double() * c["s_res"][a:b].double().repeat_interleave(case["g"], 1)
        rows += c["s_L"][a:b, None].double() * (c["L"][a:b].double() @ right_core)
        rows += c["s_A"][a:b, None].double() * (c["A"][a:b].double() @ right_corr)
        out += torch.exp(h @ rows.T - lse[:, None]) @ rows
        here = (targets >= a) & (targets < b)
        out[here] -= rows[targets[here] - a]
    return out * g[:, None]
