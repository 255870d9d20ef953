"""Keys and queries of any magnitude: scaled by powers of two against each other
they leave every score, and so every bit of the output, as it is."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import attn_ref as ref
from attn_cases import call, check, scale_keys, set_values, unpacked_ahead

pytestmark = pytest.mark.gpu

# requests of up to 16 query rows; more, over contexts that idle SMs share; many blocks, unpacked by the CTA; unpacked ahead
KINDS = {"few": ([(700, 1), (300, 2), (1, 1)], 8, 2, 128, 16), "split": ([(700, 60), (130, 130)], 8, 2, 128, 32),
         "here": ([(260, 130), (150, 150)], 64, 16, 64, 64), "ahead": ([(420, 210)], 96, 12, 64, 32)}


def case(kind, seed=3):
    lens, n_q, n_kv, D, page = KINDS[kind]
    c = ref.Case(lens, n_q, n_kv, D, page, seed=seed)
    assert unpacked_ahead(c) == (kind == "ahead")
    return c


def scaled(q, n):
    return (q.double() * 2.0 ** n).to(torch.bfloat16)


@pytest.mark.parametrize("n", [-60, -20, -10, -6, 12, 24, 30])
@pytest.mark.parametrize("kind", KINDS)
def test_attn_keys_of_any_magnitude(kind, n):
    c = case(kind)
    first = check(c)
    scale_keys(c, n)
    assert np.array_equal(call(c, q=scaled(c.q, -n)), first)


@pytest.mark.parametrize("n", [60, 90])
@pytest.mark.parametrize("kind", ["split", "here", "ahead"])
def test_attn_tiny_queries_over_large_keys(kind, n):
    c = case(kind, 4)
    scale_keys(c, n)
    c.q = scaled(c.q, -n)
    check(c)


@pytest.mark.parametrize("n", [-100, -70, 40, 60, 90, 110])
@pytest.mark.parametrize("heads", [8, 4])
def test_attn_few_rows_of_queries_of_any_magnitude(n, heads):
    """Rows that the products' units cannot hold are taken from the definition (one and two tiles of rows)."""
    c = ref.Case([(300, 2), (200, 4), (1, 1)], heads, 2, 64, 16, seed=6)
    scale_keys(c, n)
    c.q = scaled(c.q, -n)
    c.q[1] = 0
    check(c)


@pytest.mark.parametrize("gains", [(0.0, 0.05, 0.05), (0.0, 2.0 ** -30, 2.0 ** -30), (1e-3, 1e30, 1.0), (2.0 ** 41, 1.0, 2.0 ** 20)])
@pytest.mark.parametrize("small", [None, 1e-6, 1e6])
@pytest.mark.parametrize("kind", KINDS)
def test_attn_values_of_unequal_tiles(kind, small, gains):
    """Values whose size changes along the context, one position of each tile unlike its neighbours."""
    c = case(kind, 8)
    for r, (S, _) in enumerate(c.lens):
        gain = np.repeat(gains, -(-S // 3))[:S]
        if small:
            gain[7::128] = small
        set_values(c, r, np.random.default_rng(r).standard_normal((S, c.n_kv, c.D)).clip(-3, 3) * gain[:, None, None])
    check(c)


@pytest.mark.parametrize("kind", KINDS)
def test_attn_keys_of_unequal_magnitude(kind):
    """A few positions with keys 2^12 times larger or smaller than their neighbours':
    the others' scores are as exact as without them."""
    c = case(kind, 5)
    powers = np.zeros(max(s for s, _ in c.lens))
    powers[5::70], powers[17::90] = 12, -12
    scale_keys(c, powers)
    check(c, scale=0.02)
