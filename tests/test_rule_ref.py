"""The routing rules' reference against cases by hand, and what the library refuses without a device."""
import ctypes

import numpy as np
import pytest

import quantized_sparse_moe_router_gb300 as fw
import rule_ref


def test_by_hand():
    z = np.log(np.array([[1.0, 2.0, 4.0, 1.0, 3.0, 5.0]]))  # softmax: sixteenths
    ids, gates, _ = rule_ref.choose(z, 2, "softmax", renorm=False)
    assert ids.tolist() == [[5, 2]] and np.allclose(gates, [[5 / 16, 4 / 16]])
    ids, gates, _ = rule_ref.choose(z, 2, "softmax", n_group=3, top_group=1, renorm=True, scale=2.0)  # groups' sums: 3, 5, 8
    assert ids.tolist() == [[5, 4]] and np.allclose(gates, [[2 * 5 / 8, 2 * 3 / 8]])
    ids, gates, _ = rule_ref.choose(z, 2, "sigmoid", bias=np.array([1.0, 0, 0, 0, 0, 0]))  # s = w / (1 + w); the bias moves the choice alone
    assert ids.tolist() == [[0, 5]] and np.allclose(gates, np.array([[1 / 2, 5 / 6]]) / (1 / 2 + 5 / 6))


def test_ties_go_to_the_lower():
    ids, _, far = rule_ref.choose(np.zeros((1, 8)), 3, "sigmoid", n_group=4, top_group=2)
    assert ids.tolist() == [[0, 1, 2]] and far[0] == 0


def test_a_rule_needs_a_layer():
    fw.build()
    rule = fw.FwMoeRouting(0, 1, 1, 1, 1.0, None)
    for handle in (None, 777):
        assert fw.lib().fw_moe_set_routing(handle, ctypes.byref(rule), None) == fw.FW_EINVAL and "not a live handle" in fw.fw_moe_last_error()


@pytest.mark.parametrize("n_group", [1, 2, 4, 8, 16, 32])
def test_group_of_an_expert_by_multiplication(n_group):
    """e / size as the kernel takes it, for every size of group up to 256 experts."""
    for E in range(n_group, 257, n_group):
        size = E // n_group
        per = (65536 + size - 1) // size
        assert all(e * per >> 16 == e // size for e in range(256))
