"""The sequence losses from their definition, in binary64 on the host: one
sequence after another, one position after another."""
import math

import numpy as np


def _aggregate(values, mode):
    return sum(values) if mode == "sum" or not values else sum(values) / len(values)


def targets_of(offsets, tokens, n):
    """Each sequence's target positions (offsets clamped to the array)."""
    out = []
    for lo, hi in zip(offsets[:-1], offsets[1:]):
        lo = min(max(int(lo), 0), n)
        hi = max(lo, min(int(hi), n))
        out.append([t for t in range(lo, hi) if tokens is None or tokens[t] >= 0])
    return out


def policy(lp, old, ref, adv, per_token, tokens, offsets, low, high, coef, mode, d_loss, kept):
    """loss, kl, clipped, d_logprob (which starts as `kept`)."""
    n, seqs = len(lp), targets_of(offsets, tokens, len(lp))
    loss, kl, clipped, grad = [], [], [], np.array(kept, np.float64)
    for b, (lo, hi) in enumerate(zip(offsets[:-1], offsets[1:])):
        lo = min(max(int(lo), 0), n)
        grad[lo:max(lo, min(int(hi), n))] = 0.0
        terms, ks, cuts = [], [], 0
        w = 1.0 if mode == "sum" or not seqs[b] else 1.0 / len(seqs[b])
        for t in seqs[b]:
            a = float(adv[t] if per_token else adv[b])
            d = float(lp[t]) - float(old[t])
            r = math.exp(d) if d < 709 else math.inf
            border = 1.0 + high if a > 0 else 1.0 - low
            cut = (a > 0 and r > border) or (a < 0 and r < border)
            cuts += cut
            term, slope = (-border * a, 0.0) if cut else (-r * a, -r * a)
            if ref is not None:
                x = float(ref[t]) - float(lp[t])
                e = math.expm1(x) if x < 709 else math.inf
                k = math.inf if x == math.inf else e - x
                ks.append(k)
                if coef:
                    term, slope = term + coef * k, slope - coef * e
            terms.append(term)
            grad[t] = float(d_loss[b]) * w * slope
        loss.append(_aggregate(terms, mode))
        kl.append(_aggregate(ks, mode))
        clipped.append(cuts)
    return np.array(loss), np.array(kl), np.array(clipped), grad


def _softplus(v):
    return max(v, 0.0) + math.log1p(math.exp(-abs(v)))


def _sigmoid(v):
    return 1.0 / (1.0 + math.exp(-v)) if v > -700 else 0.0


def preference(lp, ref, tokens, offsets, pairs, kind, beta, margin, smoothing, mode, d_loss, kept):
    """loss, reward, d_logprob (which starts as `kept`)."""
    n, seqs = len(lp), targets_of(offsets, tokens, len(lp))
    s = [_aggregate([float(lp[t]) - (0.0 if ref is None else float(ref[t])) for t in q], mode)
         for q in seqs]
    reward = [beta * v for v in s]
    grad = np.array(kept, np.float64)
    loss = []
    for p in range(pairs):
        h = reward[p] - reward[p + pairs] - margin
        if kind == "sigmoid":
            loss.append((1 - smoothing) * _softplus(-h) + (smoothing * _softplus(h) if smoothing else 0.0))
            slope = smoothing * _sigmoid(h) - (1 - smoothing) * _sigmoid(-h)
        elif kind == "hinge":
            loss.append(max(0.0, 1.0 - h))
            slope = -1.0 if h < 1.0 else 0.0
        else:
            loss.append(((h - 0.5) / beta) ** 2)
            slope = 2.0 * (h - 0.5) / beta ** 2
        for b, sign in ((p, 1.0), (p + pairs, -1.0)):
            lo = min(max(int(offsets[b]), 0), n)
            grad[lo:max(lo, min(int(offsets[b + 1]), n))] = 0.0
            w = 1.0 if mode == "sum" or not seqs[b] else 1.0 / len(seqs[b])
            for t in seqs[b]:
                grad[t] = sign * float(d_loss[p]) * slope * beta * w
    return np.array(loss), np.array(reward), grad
