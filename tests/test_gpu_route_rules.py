"""Routing rules (softmax or sigmoid scores, selection bias, groups, gates renormalised or not) against 64 bits, on every
path of the router, and the experts behind them against the oracle."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import oracle
import quantized_sparse_moe_router_gb300 as fw
import rule_ref
import synth
from layer_inputs import GATE_TOL, DeviceLayer, OracleLayer, to_device_bf16, tolerance

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def bias_of(E, seed=0, size=0.05):
    return (np.random.default_rng(seed).normal(size=E) * size).astype(np.float32)


def set_rule(layer, rule):
    layer.set_routing(**{k: torch.from_numpy(v).to(DEV) if k == "bias" else v for k, v in rule.items()})


def route_and_check(w, layer, x, z, rule):
    T = x.shape[0]
    gates = torch.empty((T, w.k), dtype=torch.float32, device=DEV)
    ids, _ = layer.route(to_device_bf16(x, DEV), gates=gates)
    want, want_gates, _ = rule_ref.choose(z, w.k, **rule)
    assert np.array_equal(ids.cpu().numpy(), want)
    assert np.abs(gates.cpu().numpy() - want_gates).max() <= GATE_TOL * rule.get("scale", 1.0)
    off, perm, inv = layer.permutation(T)
    for got, ref in zip((off, perm, inv), oracle.permutation(want, w.E)):
        assert np.array_equal(got.cpu().numpy(), ref)
    layer.status()
    return want, want_gates


RULES = [
    dict(score="sigmoid", n_group=8, top_group=4, renorm=True, scale=2.5, bias=True),
    dict(score="softmax", n_group=1, top_group=1, renorm=False, scale=1.0),
    dict(score="softmax", n_group=8, top_group=3, renorm=False, scale=16.0, bias=True),
    dict(score="sigmoid", n_group=4, top_group=1, renorm=True, scale=1.0, bias=True),
    dict(score="sigmoid", n_group=1, top_group=1, renorm=False, scale=1.0, bias=True),
]


@pytest.mark.parametrize("E, k", [(256, 8), (64, 6), (8, 2), (40, 5), (160, 6), (128, 16), (32, 1)])
@pytest.mark.parametrize("rule", RULES)
def test_choice(E, k, rule):
    """One token, a few (the last CTA of the decode router), many (tensor-core router with and without a split of H, tiled router)."""
    n, top = rule["n_group"], rule["top_group"]
    while E % n or top * (E // n) < k:
        n, top = (n // 2, top) if top <= n // 2 else (n, top + 1) if top < n else (1, 1)
    rule = dict(rule, n_group=n, top_group=top)
    if rule.pop("bias", False):
        rule["bias"] = bias_of(E)
    w = synth.WORKLOADS["tiny"].with_(E=E, k=k, T=300, sigma_router=0.1)
    dl = DeviceLayer(w, 0, DEV)
    x = rule_ref.hidden(w, 0, dl.Wr, dl.bias, rule, 300)
    z = oracle.router_logits(x, dl.Wr, dl.bias)
    layer = dl.make(T_max=300)
    set_rule(layer, rule)
    for T in (1, 2, 5, 16, 17, 33, 300):
        route_and_check(w, layer, x[:T], z[:T], rule)
    layer.close()


def test_choice_of_many_tokens():
    """More 128-token tiles than a split of H leaves room for."""
    rule = dict(score="sigmoid", n_group=8, top_group=4, scale=2.5, bias=bias_of(64))
    w = synth.WORKLOADS["tiny"].with_(E=64, k=6, T=12000, sigma_router=0.1)
    dl = DeviceLayer(w, 0, DEV)
    x = rule_ref.hidden(w, 0, dl.Wr, dl.bias, rule, w.T)
    layer = dl.make(T_max=w.T)
    set_rule(layer, rule)
    route_and_check(w, layer, x, oracle.router_logits(x, dl.Wr, dl.bias), rule)
    layer.close()


@pytest.mark.parametrize("E, k, n_group", [(16, 4, 2), (48, 6, 4), (144, 8, 9), (208, 8, 8), (240, 4, 16)])
def test_choice_of_ragged_tiles(E, k, n_group):
    """Experts that fill a pair's tile to a half, tokens around a pair's 256."""
    rule = dict(score="softmax", n_group=n_group, top_group=2, renorm=False, bias=bias_of(E, size=0.001))
    w = synth.WORKLOADS["tiny"].with_(E=E, k=k, T=520, sigma_router=0.1)
    dl = DeviceLayer(w, 0, DEV)
    x = rule_ref.hidden(w, 0, dl.Wr, dl.bias, rule, w.T)
    z = oracle.router_logits(x, dl.Wr, dl.bias)
    layer = dl.make(T_max=w.T)
    set_rule(layer, rule)
    for T in (129, 255, 256, 257, 520):
        route_and_check(w, layer, x[:T], z[:T], rule)
    layer.close()


@pytest.mark.parametrize("T", [1, 7, 50])
@pytest.mark.parametrize("E, k, n_group, top_group", [(64, 8, 8, 2), (48, 12, 16, 4), (32, 4, 32, 4), (256, 16, 32, 3)])
def test_ties_go_to_the_lowest(T, E, k, n_group, top_group):
    """All logits equal: the first groups, their first experts; with one expert raised, it leads."""
    w = synth.WORKLOADS["tiny"].with_(E=E, k=k, T=T)
    dl = DeviceLayer(w, 0, DEV, Wr=np.zeros((E, w.H), np.float32))
    layer = dl.make(T_max=max(T, 17))
    x = to_device_bf16(synth.hidden_bf16_bits(w, 0), DEV)
    layer.set_routing("sigmoid", n_group, top_group)
    assert layer.route(x)[0].cpu().numpy().tolist() == [list(range(k))] * T
    bias = torch.zeros(E, device=DEV)
    bias[E - 1] = 1.0
    layer.set_routing("sigmoid", n_group, top_group, bias=bias)
    size = E // n_group
    rest = [e for g in list(range(top_group - 1)) + [n_group - 1] for e in range(g * size, (g + 1) * size) if e != E - 1]
    ids = layer.route(x)[0].cpu().numpy().tolist()
    if size == 1:
        rest = list(range(top_group - 1))
    assert ids == [([E - 1] + rest)[:k]] * T
    layer.close()


@pytest.mark.parametrize("T", [1, 9, 40])
def test_experts_ruled_out_and_infinite_scores(T):
    """A bias of -inf takes experts out of the choice as long as there are others; NaN logits choose nothing twice."""
    E, k = 64, 6
    w = synth.WORKLOADS["tiny"].with_(E=E, k=k, T=T, sigma_router=0.1)
    dl = DeviceLayer(w, 0, DEV)
    bias = np.zeros(E, np.float32)
    bias[::2] = -np.inf
    bias[32:] = -np.inf
    rule = dict(score="sigmoid", n_group=4, top_group=2, bias=bias)
    x = synth.hidden_bf16_bits(w, 0)
    layer = dl.make(T_max=max(T, 17))
    set_rule(layer, rule)
    ids = layer.route(to_device_bf16(x, DEV))[0].cpu().numpy()
    assert (ids % 2 == 1).all() and (ids < 32).all()
    bad = to_device_bf16(x, DEV)
    bad[0, 0] = float("nan")
    for score in ("sigmoid", "softmax"):
        layer.set_routing(score, 4, 2)
        gates = torch.empty((T, k), device=DEV)
        ids = layer.route(bad, gates=gates)[0].cpu().numpy()
        assert all(len(set(r)) == k and min(r) >= 0 and max(r) < E for r in ids.tolist())
        assert torch.isnan(gates[0]).all() and torch.isfinite(gates[1:]).all()
    layer.close()


FORWARD = [dict(score="sigmoid", n_group=4, top_group=2, scale=2.5, bias=True), dict(score="softmax", renorm=False, scale=1.0)]


@pytest.mark.parametrize("T, q8", [(1, False), (1, True), (3, False), (16, False), (16, True), (17, False), (200, False)])
@pytest.mark.parametrize("S", [0, 1])
@pytest.mark.parametrize("rule", FORWARD)
def test_forward(T, q8, S, rule):
    """Route and experts in one call and in two: the same bits, within the oracle's tolerance; and the default step is as it was afterwards."""
    w = synth.WORKLOADS["tiny"].with_(E=16, k=4, S=S, T=T, sigma_router=0.1)
    rule = {k: bias_of(16) if k == "bias" else v for k, v in rule.items()}
    dl, ol = DeviceLayer(w, 0, DEV), OracleLayer(w, 0)
    layer = dl.make(T_max=max(T, 20), act_q8=q8)
    x = rule_ref.hidden(w, 0, dl.Wr, dl.bias, rule, T)
    xd = to_device_bf16(x, DEV)
    before = layer.forward(xd)
    set_rule(layer, rule)
    gates = torch.empty((T, w.k), device=DEV)
    ids, out = layer.forward(xd, gates=gates)
    want, want_gates, _ = rule_ref.choose(oracle.router_logits(x, dl.Wr, dl.bias), w.k, **rule)
    assert np.array_equal(ids.cpu().numpy(), want)
    assert np.abs(gates.cpu().numpy() - want_gates).max() <= GATE_TOL * rule["scale"]
    ref = oracle.moe_experts(x, want, want_gates, *ol.lists_for(want), E=w.E, S=S, act_q8=q8)
    assert np.abs(out.double().cpu().numpy() - ref).max() <= tolerance(ref)
    for got, ref in zip(layer.permutation(T), oracle.permutation(want, w.E)):
        assert np.array_equal(got.cpu().numpy(), ref)
    again, _ = layer.route(xd)
    assert torch.equal(again, ids) and torch.equal(layer.ffn(xd), out)
    layer.status()
    layer.set_routing(score=None)
    after = layer.forward(xd)
    assert all(torch.equal(a, b) for a, b in zip(before, after))
    layer.close()


@pytest.mark.parametrize("T", [1, 8, 64])
def test_graph_keeps_its_rule_and_reads_the_bias_set_last(T):
    w = synth.WORKLOADS["tiny"].with_(E=16, k=2, T=T, sigma_router=0.1)
    dl = DeviceLayer(w, 0, DEV)
    layer = dl.make(T_max=max(T, 17))
    first, second = (torch.from_numpy(bias_of(16, s, 0.5)).to(DEV) for s in (1, 2))
    layer.set_routing("sigmoid", 4, 2, bias=first)
    x = to_device_bf16(synth.hidden_bf16_bits(w, 0), DEV)
    out, ids = torch.empty_like(x), torch.empty((T, 2), dtype=torch.int32, device=DEV)
    graph = fw.MoEGraph([layer], [x], [out], [ids])
    for bias in (first, second, first):
        layer.set_routing("sigmoid", 4, 2, bias=bias)
        want = layer.forward(x)
        graph.launch()
        torch.cuda.synchronize()
        assert torch.equal(ids, want[0]) and torch.equal(out, want[1])
    graph.close()
    layer.close()


def test_refusals():
    w = synth.WORKLOADS["tiny"].with_(E=24, k=4, T=2)
    dl = DeviceLayer(w, 0, DEV)
    layer = dl.make(T_max=2)
    x = to_device_bf16(synth.hidden_bf16_bits(w, 0), DEV)
    want = layer.forward(x)[0]
    for bad in (dict(n_group=0), dict(n_group=5), dict(n_group=48), dict(top_group=0), dict(top_group=2), dict(n_group=8, top_group=1), dict(scale=0.0),
                dict(scale=float("nan")), dict(scale=float("inf"))):
        with pytest.raises(fw.FwError, match="fw_moe_set_routing"):
            layer.set_routing(**bad)
    for bad in (dict(score="relu"), dict(bias=torch.zeros(24)), dict(bias=torch.zeros(23, device=DEV)), dict(bias=torch.zeros(24, device=DEV).half())):
        with pytest.raises(ValueError):
            layer.set_routing(**bad)
    assert torch.equal(layer.forward(x)[0], want)  # (none of them changed anything)
    layer.route(x)
    layer.set_routing("sigmoid")
    with pytest.raises(fw.FwError, match="FW_ESTATE"):
        layer.ffn(x)
    layer.close()
