"""The routing rules in 64 bits, from their definition, and hidden states that no choice hangs on a rounding of."""
import numpy as np

import oracle
import synth


def scores(z, score):
    if score == "sigmoid":
        return 1.0 / (1.0 + np.exp(-z))
    e = np.exp(z - z.max(1, keepdims=True))
    return e / e.sum(1, keepdims=True)


def group_scores(c, n_group):
    part = np.sort(c.reshape(c.shape[0], n_group, -1), 2)[:, :, ::-1]
    return part[:, :, :2].sum(2)


def choose(z, k, score="softmax", n_group=1, top_group=1, renorm=True, scale=1.0, bias=None):
    """-> ids [T, k], gates [T, k], and how far each token's choices are from a tie."""
    s = scores(z, score)
    c = s if bias is None else s + bias
    g = group_scores(c, n_group)
    order = np.argsort(-g, 1, kind="stable")
    kept = np.zeros_like(g, dtype=bool)
    np.put_along_axis(kept, order[:, :top_group], True, 1)
    open_ = np.where(np.repeat(kept, c.shape[1] // n_group, 1), c, -np.inf)
    ids = np.argsort(-open_, 1, kind="stable")
    best = np.take_along_axis(open_, ids, 1)[:, :k + 1]
    with np.errstate(invalid="ignore"):
        far = np.nanmin(np.where(np.isnan(best[:, :-1] - best[:, 1:]), np.inf, best[:, :-1] - best[:, 1:]), 1) if best.shape[1] > 1 else np.full(len(z), np.inf)
    if top_group < n_group:
        gs = np.take_along_axis(g, order, 1)
        far = np.minimum(far, gs[:, top_group - 1] - gs[:, top_group])
    ids = ids[:, :k].astype(np.int32)
    w = np.take_along_axis(s, ids, 1)
    return ids, scale * (w / (w.sum(1, keepdims=True) + 1e-20) if renorm else w), far / np.abs(c).max(1)


def hidden(w, layer, Wr, bias, rule, T):
    """x [T, H] bf16 bits; tokens with a choice closer than 1e-4 of the scores are drawn anew."""
    x = synth.hidden_bf16_bits(w, layer, T)
    bad, r = np.arange(T), 0
    while True:
        far = choose(oracle.router_logits(x[bad], Wr, bias), w.k, **rule)[2]
        bad = bad[far < 1e-4]
        if not len(bad):
            return x
        r += 1
        assert r < 200
        for t in bad:
            x[t] = synth.hidden_row_bf16_bits(w, layer, int(t), r)
