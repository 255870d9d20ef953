"""Routing rules where single logits of a token are NaN or infinite, against 64 bits: a NaN ranks below every number
and takes no part in the softmax or in its group's score; an infinite logit has the limit of the scores."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import oracle
import synth
from layer_inputs import GATE_TOL, DeviceLayer, to_device_bf16

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
CLEAR = 1e-4  # choices that hang on less than this of a token's largest score are left out


def scores(z, score):
    """Of one token's logits: NaN where the logit is one."""
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            return 1.0 / (1.0 + np.exp(-z))
    s, there = np.full(len(z), np.nan), ~np.isnan(z)
    if there.any():
        v = z[there]
        with np.errstate(invalid="ignore"):
            e = np.where(v == v.max(), 1.0, np.exp(v - v.max()))
        s[there] = e / e.sum()
    return s


def choose(z, k, score, n_group, top_group, renorm, bias):
    """-> ids, gates and how far one token's choices are from a tie."""
    s = scores(z, score)
    c, size = s + bias, len(z) // n_group
    group = []
    for g in range(n_group):
        best = sorted((v for v in c[g * size:(g + 1) * size] if not np.isnan(v)), reverse=True)[:2]
        group.append(sum(best) if best else -np.inf)
    order = sorted(range(n_group), key=lambda g: (-group[g], g))
    open_ = [e for g in order[:top_group] for e in range(g * size, (g + 1) * size)]
    rank = sorted(open_, key=lambda e: (np.isnan(c[e]), -c[e] if not np.isnan(c[e]) else 0.0, e))
    best = [c[e] for e in rank[:k + 1] if not np.isnan(c[e])]
    gaps = [a - b for a, b in zip(best, best[1:])]
    if top_group < n_group:
        gaps.append(group[order[top_group - 1]] - group[order[top_group]])
    w = s[rank[:k]]
    return rank[:k], w / (w.sum() + 1e-20) if renorm else w, min(gaps, default=np.inf)


def check(layer, x, z, k, rule, bias):
    T = len(x)
    layer.set_routing(bias=torch.from_numpy(bias).to(DEV), **rule)
    gates = torch.empty((T, k), dtype=torch.float32, device=DEV)
    ids = layer.route(to_device_bf16(x, DEV), gates=gates)[0].cpu().numpy()
    gates = gates.cpu().numpy()
    clear = 0
    for t in range(T):
        want, want_gates, far = choose(z[t], k, bias=bias.astype(np.float64), **rule)
        if far < CLEAR:
            continue
        clear += 1
        assert ids[t].tolist() == want, t
        assert np.array_equal(np.isnan(gates[t]), np.isnan(want_gates))
        assert np.nan_to_num(np.abs(gates[t] - want_gates)).max() <= GATE_TOL
    assert clear >= 0.6 * T
    layer.status()


@pytest.mark.parametrize("T", [1, 5, 16, 40, 300])
@pytest.mark.parametrize("E, k, n_group, top_group", [(64, 6, 8, 3), (256, 8, 8, 4), (40, 5, 4, 2), (160, 6, 5, 2), (8, 2, 4, 2), (32, 4, 16, 6)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_some_logits_are_nan(T, E, k, n_group, top_group, score):
    """One, all but one, and all of a group's logits; with groups and without."""
    size = E // n_group
    rb = synth.router_bias_f32(synth.WORKLOADS["tiny"].with_(E=E, k=k, T=T), 0)
    rb = np.zeros(E, np.float32) if rb is None else rb.copy()
    rb[1] = np.nan
    rb[2 * size + 1:3 * size] = np.nan          # one of the group is left
    rb[(n_group - 1) * size:] = np.nan          # none is
    w = synth.WORKLOADS["tiny"].with_(E=E, k=k, T=T, sigma_router=0.1)
    dl = DeviceLayer(w, 0, DEV, bias=rb)
    x = synth.hidden_bf16_bits(w, 0)
    z = oracle.router_logits(x, dl.Wr, dl.bias)
    assert np.isnan(z).any() and not np.isnan(z).all()
    bias = (np.random.default_rng(1).normal(size=E) * (0.05 if score == "sigmoid" else 0.5 / E)).astype(np.float32)
    layer = dl.make(T_max=max(T, 17))
    for groups in (dict(n_group=n_group, top_group=top_group), dict(n_group=1, top_group=1)):
        for renorm in (True, False):
            check(layer, x, z, k, dict(score=score, renorm=renorm, **groups), bias)
    layer.close()


@pytest.mark.parametrize("T", [1, 9, 64])
def test_fewer_numbers_than_experts_to_choose(T):
    """The numbers first, then the NaN ones by their ids; only their gates are NaN where gates are not made to add up."""
    E, k = 32, 6
    rb = np.full(E, np.nan, np.float32)
    rb[[7, 20]] = 0.0
    w = synth.WORKLOADS["tiny"].with_(E=E, k=k, T=T, sigma_router=0.1)
    dl = DeviceLayer(w, 0, DEV, bias=rb)
    x = synth.hidden_bf16_bits(w, 0)
    layer = dl.make(T_max=max(T, 17))
    check(layer, x, oracle.router_logits(x, dl.Wr, rb), k, dict(score="softmax", n_group=1, top_group=1, renorm=False), np.zeros(E, np.float32))
    layer.close()


@pytest.mark.parametrize("T", [1, 9, 64])
@pytest.mark.parametrize("E", [64, 40])
def test_infinite_logits(T, E):
    """+inf (an expert that is always chosen) and -inf (one that has no score) among numbers."""
    k = 4
    rb = np.zeros(E, np.float32)
    rb[9], rb[3], rb[17:20] = np.inf, -np.inf, -np.inf
    w = synth.WORKLOADS["tiny"].with_(E=E, k=k, T=T, sigma_router=0.1)
    dl = DeviceLayer(w, 0, DEV, bias=rb)
    x = synth.hidden_bf16_bits(w, 0)
    z = oracle.router_logits(x, dl.Wr, rb)
    layer = dl.make(T_max=max(T, 17))
    spread = (np.random.default_rng(2).permutation(E) * 0.01).astype(np.float32)
    for score in ("softmax", "sigmoid"):
        check(layer, x, z, k, dict(score=score, n_group=1, top_group=1, renorm=False), spread)
    layer.close()
