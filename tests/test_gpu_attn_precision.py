"""How far the attention is from 64 bits, as a norm over many outputs: the
output's own rounding and the roundings that the header names, and no others.

A rounding to a unit roundoff u leaves a number off by u / sqrt(3) times 1 / m in
the mean square, m its significand in [1, 2); significands spread evenly over
their logarithm have E[1 / m^2] = (1 - 1/4) / (2 ln 2) = 0.541. Roundings of
probabilities and values are independent, so that what they add to an output is
0.541 u^2 / 3 times sum_j p_j^2 v_j^2 for each of them; a fifth more is allowed for
(significands that are not spread evenly, values rounded in blocks). The output's
rounding is what rounding the 64-bit value gives, 2 % more for the two not being
independent. Scores are fp32: what they leave is 2^-20 and below."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import attn_ref as ref
from attn_cases import call, scale_keys, set_values, unpacked_ahead

pytestmark = pytest.mark.gpu
BF16, F16 = 2.0 ** -8, 2.0 ** -11

# (requests, query heads, key heads, dims, page, unpacked ahead) and the roundings of p and v
FEW = ([(700 + 9 * i, 1) for i in range(48)], 16, 2, 128, 64, False), [BF16, BF16]
DRAFTS = ([(700 + 9 * i, 4) for i in range(24)], 16, 4, 64, 16, False), [BF16, BF16]
SPLIT = ([(900, 40), (1500, 60)], 8, 2, 128, 32, False), [BF16, BF16]
HERE = ([(500, 130), (350, 150)], 64, 16, 64, 64, False), [BF16, BF16]
AHEAD = ([(600, 210)], 96, 12, 64, 32, True), [F16]
AHEAD128 = ([(450, 220)], 96, 12, 128, 64, True), [F16]


def exact(c):
    """The output in 64 bits, and the root of sum_j p_j^2 v_j^2."""
    out, spread = [], []
    q = c.q.to("cuda").double()
    for r, (S, n) in enumerate(c.lens):
        g = c.n_q // c.n_kv
        k, v = (torch.from_numpy(x[r]).to("cuda").repeat_interleave(g, 1) for x in (c.k, c.v))
        s = torch.einsum("thd,shd->hts", q[c.starts[r]:c.starts[r + 1]], k) / c.D ** 0.5
        see = torch.arange(S, device="cuda") <= torch.arange(S - n, S, device="cuda")[:, None]
        p = s.masked_fill(~see, float("-inf")).softmax(-1)
        out.append(torch.einsum("hts,shd->thd", p, v))
        spread.append(torch.einsum("hts,shd->thd", p * p, v * v).sqrt())
    return torch.cat(out).cpu().numpy(), torch.cat(spread).cpu().numpy()


def compare(c, roundings):
    want, spread = exact(c)
    err = np.linalg.norm(call(c) - want)
    rounded = np.linalg.norm(torch.from_numpy(want).to(torch.bfloat16).double().numpy() - want)
    bound = np.sqrt(1.02 * rounded ** 2 + 1.2 * 0.541 / 3 * sum(u * u for u in roundings) * np.linalg.norm(spread) ** 2)
    assert err <= bound, (err / np.linalg.norm(want), bound / np.linalg.norm(want))
    return err


@pytest.mark.parametrize("keys", [1.0, 2.0 ** -9])
@pytest.mark.parametrize("sizes, roundings", [FEW, DRAFTS, SPLIT, HERE, AHEAD, AHEAD128], ids=["few", "drafts", "split", "here", "ahead", "ahead128"])
def test_attn_rounds_what_it_says(sizes, roundings, keys):
    *shape, ahead = sizes
    c = ref.Case(*shape, seed=11, q_gain=1.5)
    assert unpacked_ahead(c) == ahead
    if keys != 1.0:  # small keys under large queries
        scale_keys(c, int(np.log2(keys)))
        c.q = (c.q.double() / keys).to(torch.bfloat16)
    compare(c, roundings)


@pytest.mark.parametrize("keys", [1.0, 2.0 ** -9])
@pytest.mark.parametrize("sizes", [FEW[0], DRAFTS[0], ([(6000, 1), (9000, 1)], 32, 4, 128, 128, False)], ids=["few", "drafts", "long"])
def test_attn_few_rows_round_once(sizes, keys):
    """A probability times its value's scale, and nothing before."""
    c = ref.Case(*sizes[:-1], seed=13, q_gain=1.5)
    scale_keys(c, int(np.log2(keys)))
    c.q = (c.q.double() / keys).to(torch.bfloat16)
    compare(c, [BF16])


@pytest.mark.parametrize("sizes", [SPLIT[0], HERE[0]], ids=["split", "here"])
def test_attn_more_rows_round_in_f16(sizes):
    """Where the CTA unpacks its own tiles as well."""
    compare(ref.Case(*sizes[:-1], seed=14, q_gain=1.5), [F16])


@pytest.mark.parametrize("gain, roundings", [(1.0, [F16]), (2.0 ** -5, [F16]), (2.0 ** -9, [BF16, BF16]), (2.0 ** 9, [BF16, BF16])])
def test_attn_values_by_size_where_the_cta_unpacks(gain, roundings):
    c = ref.Case(*HERE[0][:-1], seed=15, q_gain=1.5)
    for r, (S, _) in enumerate(c.lens):
        set_values(c, r, gain * np.random.default_rng(r).standard_normal((S, c.n_kv, c.D)))
    compare(c, roundings)


@pytest.mark.parametrize("gain, roundings", [(1.0, [F16]), (2.0 ** -5, [F16]), (2.0 ** -9, [BF16, BF16]), (2.0 ** 9, [BF16, BF16])])
def test_attn_values_unpacked_ahead_by_size(gain, roundings):
    """f16 while a tile's largest magnitudes lie in the window that the header gives, else bf16."""
    *shape, _ = AHEAD[0]
    c = ref.Case(*shape, seed=12, q_gain=1.5)
    S = c.lens[0][0]
    set_values(c, 0, gain * np.random.default_rng(12).standard_normal((S, c.n_kv, c.D)))
    compare(c, roundings)
