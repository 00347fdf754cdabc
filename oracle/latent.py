"""Oracle of what lies around a speculative decoding step, in 64 bits on the CPU: rotation by
position, rows of a paged cache of latents, and the way from logits to probabilities.

(Attention over latents is ``oracle.spec.attention`` with one key/value head.)
"""

import numpy as np

from .spec import ancestors


def rotate(x, position, inv_freq, start, interleaved, factor):
    """One token's heads (heads, dim), the columns from ``start`` on rotated in pairs."""
    out = np.array(x, np.float64)
    half = len(inv_freq)
    for i, f in enumerate(np.asarray(inv_freq, np.float64)):
        a, b = (start + 2 * i, start + 2 * i + 1) if interleaved else (start + i, start + i + half)
        t = float(position) * f
        out[:, a] = factor * (x[:, a] * np.cos(t) - x[:, b] * np.sin(t))
        out[:, b] = factor * (x[:, b] * np.cos(t) + x[:, a] * np.sin(t))
    return out


def target_probs(logits, tokens, parents, text, prompt, temperature=1.0, repetition=1.0,
                 presence=0.0, frequency=0.0, bias=(), allowed=None):
    """One request: logits (n, vocab), its text's tokens of which the first ``prompt`` are its
    prompt, (id, value) pairs of biases, allowed (n, vocab) truth values.  tokens None: nodes do
    not count; parents None: a chain.  Returns the rows of probabilities and of x before the
    softmax."""
    n, V = logits.shape
    if parents is None:
        parents = list(range(-1, n - 1))
    on = ancestors(parents)
    out, xs = np.zeros((n, V)), np.zeros((n, V))
    in_prompt = np.zeros(V, bool)
    since = np.zeros(V, np.int64)
    for j, v in enumerate(text):
        if 0 <= v < V:
            if j < prompt:
                in_prompt[v] = True
            else:
                since[v] += 1
    for i in range(n):
        count = since.copy()
        if tokens is not None:
            for j in np.nonzero(on[i])[0]:
                if 0 <= tokens[j] < V:
                    count[tokens[j]] += 1
        x = np.array(logits[i], np.float64)
        met = in_prompt | (count > 0)
        with np.errstate(invalid="ignore"):
            x = np.where(met, np.where(x > 0, x / repetition, x * repetition), x)
            x = x - count * float(frequency) - np.where(count > 0, float(presence), 0.0)
            for v, b in bias:
                if 0 <= v < V:
                    x[v] += b
        x[np.isnan(x)] = -np.inf
        if allowed is not None:
            x[~allowed[i]] = -np.inf
        xs[i] = x
        top = x.max()
        if top == -np.inf:
            continue
        if not temperature > 0:
            out[i, int(np.argmax(x))] = 1.0
        elif top == np.inf:
            out[i] = (x == np.inf) / (x == np.inf).sum()
        else:
            w = np.exp((x - top) / temperature)
            out[i] = w / w.sum()
    return out, xs
