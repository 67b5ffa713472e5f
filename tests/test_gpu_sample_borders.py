"""lora_sample where sums of very many small weights decide: draws whose border is a small part of one such weight away."""
from decimal import Decimal, getcontext

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from heterogeneous_adapters_lora_gb300 import lora as L

pytestmark = pytest.mark.gpu

getcontext().prec = 60
V = 128256
TOP_AT = 777  # the column of the largest logit; all others are equal


def draws(top, low, temperature, seed, many):
    """Random numbers whose border among the equal columns is 1e-4 to 1e-2 of a column away, and the tokens that they choose.

    A weight is accurate to 2e-13 of itself and 2^-62 of the largest, which is exact: at 2^-26.4 of the largest, the smallest
    here, 2e-11 of itself, so 128255 of them are off by less than 1e-5 columns.
    """
    q = ((Decimal(low) - Decimal(top)) / Decimal(float(np.float32(temperature)))).exp()
    total = 1 + (V - 1) * q
    r = np.random.RandomState(seed)
    first = 1 - float((V - 1) * q / total)  # below it the first column is drawn
    us, tokens = [], []
    for _ in range(200000):
        u = np.float32(r.uniform(first, 1.0))
        at = (Decimal(float(u)) * total - 1) / q  # in columns
        if u >= 1 or at < 0:
            continue
        whole = int(at)
        part = at - whole
        if min(part, 1 - part) < Decimal("1e-4") or min(part, 1 - part) > Decimal("1e-2"):
            continue
        column = whole if whole < TOP_AT else whole + 1
        us.append(float(u))
        tokens.append(column)
        if len(us) == many:
            return us, tokens
    raise AssertionError("no draws near a border")


@pytest.mark.parametrize("top,low,temperature", [(17.875, -0.37109375, 1.1), (16.0, 0.5, 0.85), (12.0, -0.34375, 0.85), (13.125, 0.25, 1.1),
                                                 (20.0, 0.0, 1.3), (9.5, -1.25, 0.7)])
@pytest.mark.parametrize("many", [1, 24, 200])
def test_draws_beside_borders(top, low, temperature, many):
    us, tokens = draws(top, low, temperature, many, many)
    row = torch.full((V,), low, dtype=torch.bfloat16)
    row[TOP_AT] = top
    assert float(row[0]) == low and float(row[TOP_AT]) == top
    x = row.cuda().expand(many, V).contiguous()
    got = torch.zeros(many, dtype=torch.int32, device="cuda")
    L.lora_sample(x, V, many, V, torch.full((many,), temperature, device="cuda"), None, None, None, torch.tensor(us, device="cuda"), got, None)
    assert got.tolist() == tokens
