"""Filters whose border lies between two values that a logit can have, or next to one (tolerances: test_gpu_sample.py)."""
import numpy as np
import pytest
import torch

from tests.test_gpu_sample import check, make, place, requests, run

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


# (T, largest logit, two neighbouring floats the first below the second, min_p): as the weights are computed, the first's is at least
# min_p and the second's is not, for they are within 2^-31 of themselves, and the logits are nearer to each other.
STEPS_BACK = [(t, float.fromhex(m), float.fromhex(a), float.fromhex(b), float.fromhex(mp)) for t, m, a, b, mp in [
    (float.fromhex("0x1.03bp+0"), "0x1.15814ep-2", "-0x1.deb2p-11", "-0x1.deb1fep-11", "0x1.879caep-1"),
    (float.fromhex("0x1.044p+0"), "0x1.9cd9f4p-1", "-0x1.37fp-13", "-0x1.37effep-13", "0x1.cf3156p-2"),
    (float.fromhex("0x1.0f1p+0"), "0x1.adb90ap+1", "0x1.abp-15", "0x1.ab0002p-15", "0x1.57e28p-5"),
    (float.fromhex("0x1.109p+0"), "0x1.5fdd2cp+2", "0x1.aebffep-12", "0x1.aecp-12", "0x1.770244p-8"),
    (float.fromhex("0x1.176p+0"), "0x1.93a16ap+2", "-0x1.e35p-10", "-0x1.e34ffep-10", "0x1.948b7cp-9"),
    (float.fromhex("0x1.1a9p+0"), "0x1.46f14ep-3", "0x1.d96f6p-8", "0x1.d96f62p-8", "0x1.bdf69cp-1")]]


@pytest.mark.parametrize("V,p", [(3, 1.0), (400, 1.0), (5003, 1.0), (5003, 0.99999994), (100000, 0.99999994)])
def test_weights_that_step_back(ss, V, p):
    """Whichever of the two are kept, they are the ranking's first, the draw is one of them, and every way says the same."""
    rows = len(STEPS_BACK)
    x = torch.full((rows, V), -200.0, device="cuda")
    for r, (_, m, a, b, _) in enumerate(STEPS_BACK):
        x[r, 0], x[r, 1], x[r, 2] = m, a, b
    T, mp = [s[0] for s in STEPS_BACK], [s[4] for s in STEPS_BACK]
    u = torch.full((rows,), 1.0 - 2.0 ** -24, device="cuda")
    check(ss, x, T=T, mp=mp, p=p, u=u)
    few, wide = (ss.Filter(*requests(rows, T, None, q, mp)) for q in (None, p))
    assert torch.equal(run(ss, x[:, :3].contiguous(), few, u)[2], run(ss, x, wide, u)[2])


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("V", [50, 5003, 100000])
def test_min_p_below_the_weights_steps(ss, kind, V):
    """Logits whose weights are rounded to nothing are kept down to min_p, and not drawn."""
    x = torch.full((6, V), -90.0, device="cuda")
    x[:, 3:20], x[:, 20:30], x[:, 30:40], x[:, 1] = -40.0, -50.0, -34.0, 0.0
    x[5] = place(x[5:6], 0, 0) * 1e4
    x = place(x.to({"bf16": torch.bfloat16, "f32": torch.float32}[kind]), 1, 1)
    kw = dict(T=[1.0, 1.0, 2.0, 1.0, 1.0, 1e4], mp=[1e-20, 1e-17, 1e-30, 1e-38, 1e-45, 1e-20], u=torch.full((6,), 1.0 - 2.0 ** -24, device="cuda"))
    check(ss, x, **kw)
    check(ss, x, p=0.99999994, **kw)


def test_the_last_weights_count(ss):
    """Weights of one step of 2^-44, at the least logit that has one: of many, rows of either type have the same sums."""
    V = 240001
    x = torch.full((2, V), -31.25, device="cuda")
    x[:, 0], x[:, 1:40001] = 0.0, -21.25
    f = ss.Filter(*requests(2, float.fromhex("0x1.007aa8p+0"), None, 0.99999994, None))
    u = torch.tensor([0.3, 0.9999999], device="cuda")
    got = [run(ss, x.to(t), f, u) for t in (torch.bfloat16, torch.float32)]
    assert got[0][2].tolist() == [39923] * 2  # the first sums that reach (1 - 2^-24) of the total, by hand
    for a, b in zip(*(g[:3] for g in got)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("V,p", [(300, 1.0), (5003, 1.0), (5003, 0.999)])
def test_min_p_of_one_keeps_the_largest_alone(ss, kind, V, p):
    """And those equal to it, though the others' weights are 1 in any arithmetic: at high temperatures, and among tiny logits."""
    x = make(5, V, kind, seed=V)
    x[2:] = (x[2:].float() * 1e-20).to(x.dtype)
    x[4, 5::7] = x[4].max()
    check(ss, x, T=[1e12, 1e35, 1.0, 0.3, 1.0], mp=[1.0, 7.0, 1.0, 1.0, 1.0], p=p)
