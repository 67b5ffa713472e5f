"""lora_sample where several CTAs share a row: parts that hold nothing, odd numbers in one part alone, equals over all."""
import math

import pytest

torch = pytest.importorskip("torch")

from test_gpu_sample import check, rows, uniform

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,V", [(1, 40001), (2, 47999), (3, 48001), (39, 96009), (77, 100003), (153, 40000), (310, 40008)])
def test_rows_and_lengths(T, V):
    """From one row of eight CTAs to more rows than find room at once."""
    u = uniform(T, V)
    check(rows(T, V, V + T), [(0.6, 1.0, 0.0)[t % 3] for t in range(T)], [(0, 50, 0, 3000)[t % 4] for t in range(T)],
          [(1.0, 0.95)[t % 2] for t in range(T)], [(0.0, 0.0, 0.0, 0.01, 0.2)[t % 5] for t in range(T)], u)


def odd_rows(V, seed):
    x = rows(20, V, seed)
    last = V - 5
    x[1] = -math.inf
    x[2] = math.nan
    x[3, 1:] = -math.inf            # one column, in the first part
    x[4, :last] = -math.inf         # a few, in the last
    x[5, : V // 2] = math.nan
    x[6, last] = math.inf
    x[7, ::9973] = math.inf
    x[8] = 0.0
    x[8, 1::2] = -0.0
    x[9] = 3.0                      # all equal
    x[10, 7] = 2.0 ** -55           # at the border of the range that is counted at once, one part alone
    x[11, last] = -(2.0 ** -55)
    x[12, V // 3] = 1e-30
    x[13, last] = 600.0             # above that range
    x[14, 11] = -600.0              # below it, and of no weight
    x[15] = torch.finfo(torch.bfloat16).min
    x[16, ::2] = torch.finfo(torch.bfloat16).min
    x[17] = -600.0                  # below it, all of them
    x[17, last] = -599.0
    x[18, : V - 9] = -math.inf      # nothing but the last vector that is not whole
    x[19] *= 1e4
    return x


@pytest.mark.parametrize("V", [40003, 50001, 128259])
def test_odd_rows(V):
    x = odd_rows(V, V)
    T = x.shape[0]
    check(x, uniform=uniform(T, 1))
    check(x, [0.0] * T, uniform=uniform(T, 2))
    check(x, [3.0] * T, [1 + 700 * t for t in range(T)], [0.97] * T, [1e-4] * T, uniform(T, 3))
    check(x, [300.0] * T, None, [0.5] * T, None, uniform(T, 4))


@pytest.mark.parametrize("V", [40000, 128256])
def test_equals_end_where_a_part_ends(V):
    """Weights of exactly 1: the chosen index is floor(u n), at and beside the borders of halves, quarters and eighths."""
    x = torch.zeros(16, V, dtype=torch.bfloat16)
    borders = [V // 8, V // 4, V // 2, 3 * V // 4]
    k = [b + d for b in borders for d in (-1, 0, 1, 9)]
    check(x, top_k=k, uniform=[1 - 2.0 ** -24] * 16)
    check(x, top_k=k, uniform=[0.5] * 16)
    check(x, top_p=[1.0, 0.5, 0.25, 0.125] * 4, uniform=[1 - 2.0 ** -24] * 16)


@pytest.mark.parametrize("T,V", [(1, 39999), (152, 39990), (153, 39990), (15, 128256), (16, 128256), (17, 128256), (20, 257024), (38, 128000), (39, 120000),
                                 (76, 100003), (76, 116001), (77, 90000),
                                 (17, 257024), (64, 128256), (76, 131000), (76, 131040), (1, 36000)])
def test_rows_in_shared_memory_or_not(T, V):
    """Sizes at and beside the ones from which a CTA no longer keeps its part of the row."""
    x = rows(T, V, T)
    x[:, 5::7] = -math.inf
    check(x, [1.0] * T, [0, 20] * (T // 2) + [3] * (T % 2), None, None, uniform(T, V))
