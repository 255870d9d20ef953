"""What the attention reports in its status word, and what it must not."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import attn_ref as ref
import quantized_sparse_moe_router_gb300 as fw
from attn_cases import DEV, call, unpacked_ahead

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens, n_q, n_kv, ahead", [([(700, 1), (650, 3)], 4, 2, False), ([(700, 90), (400, 33)], 8, 2, False),
                                                     ([(700, 210)], 96, 12, True)])
@pytest.mark.parametrize("window, sinks", [(100, 0), (77, 20), (1, 0)])
def test_pages_behind_the_window_may_be_gone(lens, n_q, n_kv, ahead, window, sinks):
    """Table entries that no row's window or kept first tokens reach are free for
    other use: -1 there, in the middle of 128 positions too, is no error."""
    c = ref.Case(lens, n_q, n_kv, 64, 16, seed=window)
    assert unpacked_ahead(c, window, sinks) == ahead
    want, tol = c.reference(window, sinks)
    table = c.table.copy()
    for r, (S, n) in enumerate(lens):
        lo = S - n + 1 - window  # the first position that a row sees beside the kept ones
        gone = np.arange(c.max_blocks)
        table[r, (gone * 16 + 16 <= lo) & (gone * 16 >= sinks)] = -1
    got = call(c, window, sinks, table=table)
    assert (np.abs(got - want) <= tol).all()
