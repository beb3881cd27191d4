"""Beam search's selection in 64 bits (numpy)."""

import numpy as np


def log_probabilities(x):
    """x [vocab] -> log-probabilities, or None where they are not defined (NaN, +inf, no finite logit)."""
    x = np.asarray(x, dtype=np.float64)
    if np.isnan(x).any() or (x == np.inf).any() or not np.isfinite(x).any():
        return None
    top = x.max()
    return x - top - np.log(np.exp(x - top).sum())


def select(logits, scores, width, finished=None, eos=-1, pad=0, history=None, lens=None):
    """logits [requests][beams][vocab] float64, scores [requests][beams]; returns a dict of arrays."""
    requests, beams, vocab = logits.shape
    out = {k: [] for k in ("scores", "parents", "tokens", "finished", "history", "lens")}
    for r in range(requests):
        found = []
        for b in range(beams):
            s = float(scores[r][b])
            if not np.isfinite(s):
                continue
            if finished is not None and finished[r][b]:
                found.append((s, b, pad, True, 0.0))
                continue
            lp = log_probabilities(logits[r, b])
            if lp is None:
                continue
            x = logits[r, b]
            # more than width of one beam cannot be chosen: the higher logit, of equal ones the lower token
            order = np.lexsort((np.arange(vocab), -x))[:width]
            found += [(s + lp[v], b, int(v), False, float(x[v])) for v in order if x[v] > -np.inf]
        found.sort(key=lambda c: (-c[0], c[1], -c[4], c[2]))
        found = found[:width] + [(-np.inf, None, pad, False, 0.0)] * (width - len(found))
        for s, b, v, was, _ in found:
            row = 0 if b is None else b
            out["scores"].append(s)
            out["parents"].append(r * beams + row)
            out["tokens"].append(v)
            out["finished"].append(was or (b is not None and v == eos))
            if history is not None:
                h = list(history[r][row])
                n = min(max(int(lens[r][row]), 0), len(h))
                if b is not None and not was and n < len(h):
                    h[n] = v
                    n += 1
                out["history"].append(h)
                out["lens"].append(n)
    return {k: np.array(v) for k, v in out.items() if v}
