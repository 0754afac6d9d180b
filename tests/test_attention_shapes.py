"""Attention where its work layout takes other ways: more segments than threads, many query heads a key head, many shares."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF, F32 = torch.bfloat16, torch.float32


def _cases():
    spec = importlib.util.spec_from_file_location("prefix_cases", os.path.join(ROOT, "tests", "test_prefix_attention.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("R,G,Hq,Hk,D", [(639, 1, 2, 1, 64), (640, 0, 2, 1, 64), (641, 0, 2, 2, 128), (1500, 3, 2, 1, 64), (700, 700, 1, 1, 64),
                                         (2600, 5, 1, 1, 128)])
def test_more_segments_than_threads(R, G, Hq, Hk, D):
    m = _cases()
    per = R // max(G, 1)
    groups = tuple((per if g < G - 1 else R - per * (G - 1), 3 + 41 * g % 300) for g in range(G))
    n = [(i * 7) % 4 for i in range(R)]  # every fourth request without rows
    kv = [(k + (i * 31) % 150) * (i % 11 > 0) for i, k in enumerate(n)]  # some without keys
    m._run(m.Case(n, kv, Hq, Hk, D, 16, BF, groups))


@pytest.mark.parametrize("per_head", [16, 32, 48, 64, 96, 128, 192, 256, 320, 512, 1024])
@pytest.mark.parametrize("D", [64, 128])
def test_many_query_heads_a_key_head(per_head, D):
    m = _cases()
    Hk = 2 if per_head <= 512 else 1
    m._run(m.Case([2, 1, 5, 3], [300, 1, 70, 900], Hk * per_head, Hk, D, 32, BF, ((2, 200), (1, 129))))


@pytest.mark.parametrize("dt,D", [(F32, 64), (BF, 40), (F32, 256)])
@pytest.mark.parametrize("n,kv", [([1], [5000]), ([1], [4095]), ([3, 1], [9000, 2200])])
def test_more_shares_of_a_row_than_lanes(dt, D, n, kv):
    m = _cases()
    m._run(m.Case(n, kv, 1, 1, D, 16, dt))
