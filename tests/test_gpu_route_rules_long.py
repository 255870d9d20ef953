"""Routing rules at hidden sizes of real layers, against 64 bits: where the router's ring of stages comes round, and where
the choice adds up more parts of H than it loads at once."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import oracle
import quantized_sparse_moe_router_gb300 as fw
import rule_ref
from layer_inputs import GATE_TOL

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def layer_of(H, E, k, T_max, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    Wr = torch.randn(E, H, generator=g, device=DEV) * 0.85 * H ** -0.5
    nothing = torch.zeros(E, 64 * H // 32 * 34, dtype=torch.uint8, device=DEV)
    return fw.MoELayer(H, 64, E, k, T_max=T_max, weights=dict(router_w=Wr, w_gate=nothing, w_up=nothing, w_down=nothing)), Wr, g


def logits(x, Wr):
    return (x.double() @ Wr.double().t()).cpu().numpy()


def tokens(T, Wr, k, rule, g):
    """x, and its logits in 64 bits; tokens whose choice hangs on less than 1e-4 of their scores are drawn anew."""
    x = torch.randn(T, Wr.shape[1], generator=g, device=DEV).bfloat16()
    z = logits(x, Wr)
    for _ in range(100):
        near = np.flatnonzero(rule_ref.choose(z, k, **rule)[2] < 1e-4)
        if not len(near):
            return x, z
        x[torch.from_numpy(near).to(DEV)] = torch.randn(len(near), Wr.shape[1], generator=g, device=DEV).bfloat16()
        z[near] = logits(x[torch.from_numpy(near).to(DEV)], Wr)
    raise AssertionError("no clear choices")


@pytest.mark.parametrize("H", [1024, 2048, 7168])
@pytest.mark.parametrize("E, k, n_group, top_group", [(256, 8, 8, 4), (160, 6, 5, 2), (64, 6, 4, 2), (16, 4, 1, 1), (40, 5, 4, 2), (8, 2, 4, 2)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_choice(H, E, k, n_group, top_group, score):
    """A token, a few, and as many as take one part of H, several, eight and sixteen."""
    sizes = (1, 2, 16, 17, 64, 300, 1024, 1100) if E != 256 else (1, 3, 16, 64, 600, 1024, 1025, 4096)
    layer, Wr, g = layer_of(H, E, k, max(sizes), H + E)
    bias = (np.random.default_rng(E).normal(size=E) * (0.02 if score == "sigmoid" else 0.02 / E)).astype(np.float32)
    rule = dict(score=score, n_group=n_group, top_group=top_group, renorm=True, scale=2.5, bias=bias)
    layer.set_routing(**dict(rule, bias=torch.from_numpy(bias).to(DEV)))
    x, z = tokens(max(sizes), Wr, k, rule, g)
    ids_all, gates_all, _ = rule_ref.choose(z, k, **rule)
    for T in sizes:
        gates = torch.full((T, k), 7.0, device=DEV)
        ids, _ = layer.route(x[:T], gates=gates)
        assert np.array_equal(ids.cpu().numpy(), ids_all[:T]), T
        assert np.abs(gates.double().cpu().numpy() - gates_all[:T]).max() <= GATE_TOL * 2.5, T
        for got, want in zip(layer.permutation(T), oracle.permutation(ids_all[:T], E)):
            assert np.array_equal(got.cpu().numpy(), want), T
        again = torch.empty_like(gates)
        assert torch.equal(layer.route(x[:T], gates=again)[0], ids) and torch.equal(again, gates)
    layer.status()
    layer.close()
