"""Float64 oracle of learning through a packed head: the gradient of the
cross-entropy with respect to the hidden states, the clipped policy loss and
the preference loss.  Plain loops over tokens and sequences from the formulas;
independent of the CUDA library."""
import numpy as np

from .archead_oracle import bf16_decode, dequantized_factors


def dense_rows(comp, g, g_B):
    """(W_hat [V, d], entrywise sum of the absolute terms of each entry's branches)."""
    L, R, Q, A, B = dequantized_factors(comp, g, g_B)
    return L @ R + Q + A @ B, np.abs(L) @ np.abs(R) + np.abs(Q) + np.abs(A) @ np.abs(B)


def ce_gradient(W, h, lse, targets, grad_ce, rows=None):
    """dLoss/dh [T, d] of a loss with gradients grad_ce [T] with respect to
    ce[t] = lse[t] - h[t] . W[targets[t]] (rows whose gradient is 0 are zero).
    Also returns G = softmax - onehot [T, V].  targets of -1 have no row here."""
    live = np.asarray(grad_ce) != 0
    h, lse = np.where(live[:, None], h, 0.0), np.where(live, lse, 0.0)
    G = np.exp(h @ W.T - lse[:, None])
    for t in np.nonzero(live)[0]:
        if targets[t] >= 0:
            G[t, targets[t]] -= 1.0
    G[~live] = 0.0
    return (G @ W) * np.where(live, grad_ce, 0.0)[:, None], G


def hidden_f64(h_bits):
    return bf16_decode(h_bits)


def policy_loss(ce, old, adv, cu, mask=None, ref=None, clip_low=0.2, clip_high=0.2, kl_coef=0.0, reduction="tokens",
                advantage_per="token", scale=1.0):
    """(loss, dloss/dce [T], stats [3]) of the clipped policy loss."""
    ce, old, adv = (np.asarray(x, np.float64) for x in (ce, old, adv))
    T, S = ce.size, len(cu) - 1
    keep = np.ones(T, bool) if mask is None else np.asarray(mask, bool)
    counted = [[t for t in range(cu[s], cu[s + 1]) if keep[t]] for s in range(S)]
    total, alive = sum(map(len, counted)), sum(1 for c in counted if c)
    loss, grad, stats = 0.0, np.zeros(T), np.zeros(3)
    for s, tokens in enumerate(counted):
        w = {"tokens": 1.0 / max(total, 1), "sequences": 1.0 / (max(alive, 1) * max(len(tokens), 1)), "sum": 1.0}[reduction]
        for t in tokens:
            A = adv[s] if advantage_per == "sequence" else adv[t]
            with np.errstate(over="ignore"):
                r = np.exp(old[t] - ce[t])
            plain, clipped = -A * r, -A * min(max(r, 1 - clip_low), 1 + clip_high)
            cut = clipped > plain
            l, g = max(plain, clipped), 0.0 if cut else A * r
            stats[0] += cut
            stats[1] += np.expm1(old[t] - ce[t]) - (old[t] - ce[t])
            if ref is not None:
                d = ce[t] - float(ref[t])
                k = np.expm1(d) - d
                stats[2] += k
                l, g = l + kl_coef * k, g + kl_coef * np.expm1(d)
            loss += scale * w * l
            grad[t] = scale * w * g
    return loss, grad, stats / max(total, 1)


def preference_loss(ce, cu, mask=None, ref=None, beta=0.1, kind="sigmoid", label_smoothing=0.0, margin=0.0,
                    average=False, scale=1.0):
    """(loss, dloss/dce [T], rewards [2, N]) of the preference loss."""
    ce = np.asarray(ce, np.float64)
    T, N = ce.size, (len(cu) - 1) // 2
    keep = np.ones(T, bool) if mask is None else np.asarray(mask, bool)
    grad, rewards, loss = np.zeros(T), np.zeros((2, N)), 0.0
    for i in range(N):
        score, tokens = [], []
        for s in (i, N + i):
            c = [t for t in range(cu[s], cu[s + 1]) if keep[t]]
            v = sum((0.0 if ref is None else float(ref[t])) - ce[t] for t in c)
            score.append(v / max(len(c), 1) if average else v)
            tokens.append(c)
        D = score[0] - score[1]
        h = beta * D - margin
        if kind == "sigmoid":
            loss += (1 - label_smoothing) * np.logaddexp(0, -h) + label_smoothing * np.logaddexp(0, h)
            with np.errstate(over="ignore"):
                slope = beta * (label_smoothing / (1 + np.exp(-h)) - (1 - label_smoothing) / (1 + np.exp(h)))
        elif kind == "hinge":
            loss += max(0.0, 1 - h)
            slope = -beta if h < 1 else 0.0
        else:
            loss += (D - 0.5 / beta) ** 2
            slope = 2 * (D - 0.5 / beta)
        for c, sign in zip(tokens, (-1.0, 1.0)):
            for t in c:
                grad[t] = sign * slope * scale / N / (len(c) if average else 1)
        rewards[:, i] = beta * score[0], beta * score[1]
    return (scale * loss / N if N else 0.0), grad, rewards
