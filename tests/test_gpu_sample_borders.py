"""Filters whose border lies between two values that a logit can have, or next to one (tolerances: test_gpu_sample.py)."""
import numpy as np
import pytest
import torch

from tests.test_gpu_sample import check, make, place

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.fixture(scope="module")
def ss():
    from speculative_decoding_verification_35_gb300 import specsample
    return specsample


def next_to(x, m, T, side):
    """A min_p just above (side 1) or below (-1) the weight of logits x: they go, or stay."""
    return float(np.float32(np.exp((x - m) / T) * (1 + side * 1e-3)))


HELD, LYING = (6, 40000), (77, 128256)  # rows that are held, and read where they lie


@pytest.mark.parametrize("shape,hidden,more", [(HELD, h, m) for h in (-1e9, -1e4, -3.3895314e38, 1e-20)  # each has no quick bin
                                               for m in (dict(p=0.999), dict(k=3000), dict(p=0.9995, k=20000))] + [(LYING, -1e9, dict(p=0.999))])
def test_min_p_between_two_bf16(ss, shape, hidden, more):
    rows, V = shape
    x = torch.full((rows, V), 1.5, device="cuda")
    T, mp = [], []
    for r in range(rows):
        m, at, t, side = [(10.0, 7.0, 1.0, 1), (10.0, 7.0, 1.0, -1), (3.0, 2.015625, 0.7, 1), (30.0, -2.5, 6.0, 1), (-1.0, -1.0078125, 0.01, 1),
                          (12.0, 7.03125, 1.0, -1)][r % 6]
        x[r] = min(at, 0.0) - 20.0 * t
        x[r, r % 7::97] = at
        x[r, 1000 + r] = m
        T.append(t), mp.append(next_to(at, m, t, side))
    x[:, 5] = hidden
    x = place(x.to(torch.bfloat16), 3, 1)
    check(ss, x, T=T, mp=mp, **more)
    if shape == HELD:
        check(ss, x, T=T, mp=mp, out=place(torch.zeros_like(x), 2, 2), **more)


@pytest.mark.parametrize("rows,V", [(9, 30011), LYING])
def test_min_p_of_rows_outside_the_quick_bins(ss, rows, V):
    x = make(rows, V, "bf16", sigma=1.5, zipf=0.0, seed=V)
    x[:, ::5] = -1e4
    rng = np.random.default_rng(rows)
    check(ss, x, T=rng.choice([0.7, 1.0, 1.4], rows), k=rng.choice([0, 0, 4000], rows), p=rng.choice([0.99, 0.999, 0.99999], rows),
          mp=rng.uniform(0.01, 0.4, rows).astype(np.float32))


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("rows,V", [(9, 700), (9, 5003), (9, 100000), LYING])
def test_tiny_temperatures(ss, kind, rows, V):
    """Down to the least of which log2(e) / T is a float, the largest logit and those like it are all there is."""
    x = make(rows, V, kind, seed=V, pad=1)
    x[:, 7] = -1e9  # (no quick bin)
    x[2] = 0.0
    x[3, ::2], x[3, 1::2] = 0.0, -1e-45  # (bf16: zeros)
    T = [1e-37, 5e-39, 1e-38, 3e-38, 4.3e-37, 4.4e-37, 1e-36, 1e-30, 4.3e-39]
    for kw in (dict(p=0.9), dict(p=0.9, mp=0.3), dict(p=0.5, k=2000), dict()):
        check(ss, x, T=np.resize(T, rows), **kw)
