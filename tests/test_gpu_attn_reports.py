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


@pytest.mark.parametrize("lens, n_q, n_kv, max_q, starts, bad", [
    ([(60, 1), (90, 2), (33, 1)], 8, 2, 1, None, [1]),                          # more than max_q, all within the decode kernel's rows
    ([(60, 2), (90, 1), (33, 4)], 8, 2, 2, None, [2]),                          # the same past its 8-row tile
    ([(60, 30), (300, 90), (33, 1)], 8, 2, 40, None, [1]),                      # long and short requests
    ([(600, 211), (300, 200)], 96, 12, 205, None, [0]),                         # tiles unpacked ahead
    ([(60, 1), (90, 1), (33, 1), (20, 1)], 8, 2, 3, [0, 4, 1, 2, 3], [0, 1]),   # too many, then less than none; the others have rows 1 and 2
    ([(60, 1), (90, 1), (33, 1)], 8, 2, 1, [0, 1, 7, 3], [1, 2]),               # past T
    ([(60, 1), (90, 1), (33, 1)], 8, 2, 1, [-1, 1, 2, 3], [0]),                 # before row 0
    ([(60, 40), (90, 30), (33, 20)], 8, 2, 40, [0, 70, 10, 30], [0, 1]),
    ([(60, 40), (90, 30), (33, 20)], 8, 2, 60, [0, 40, 1000, 90], [1, 2])])
def test_requests_that_the_call_cannot_take_are_reported_and_not_written(lens, n_q, n_kv, max_q, starts, bad):
    c = ref.Case(lens, n_q, n_kv, 64, 16, seed=3)
    d = c.device()
    at = c.starts if starts is None else np.array(starts, np.int32)
    out = torch.full_like(d["q"], 7.0)
    word = torch.zeros(1, dtype=torch.int32, device=DEV)
    fw.attn_q4(d["q"], d["cache"], d["block_table"], torch.from_numpy(at).to(DEV), d["seq_lens"], max_q, out=out, status=word)
    got = out.double().cpu().numpy()
    assert word.item() == fw.KV_BAD_QUERIES
    written = np.zeros(c.T, bool)
    for r in range(len(lens)):
        n = at[r + 1] - at[r]
        if r in bad or n == 0:
            continue
        rows = slice(at[r], at[r + 1])
        want, tol = ref.attention(c.q.double().numpy()[rows], c.k[r], c.v[r], n, 1 / 8, 0, 0)
        assert (np.abs(got[rows] - want) <= tol).all()
        written[rows] = True
    assert (got[~written] == 7).all()
