"""Filtered distributions on the GPU against the fp64 oracle.

Tolerances. A weight is within 2^-31 of itself and rounded to 2^-44 of the largest, so a sum of n weights is within
2^-31 of itself and n 2^-45: for n <= 2^18 and sums of at least 1 that is 2^-27 at the very worst, where all roundings of
all weights go one way; the sums here (n <= 2^16 wherever the total is near 1) stay within SLACK = 2^-28. A count or a
draw may differ from the oracle's only where a border lies that near, which none of the seeds' rows does except by chance:
the oracle gives the range, mostly a single value. A log-probability is computed in double and rounded once to float: 2^-24 of
itself, and 2^-28 for the total's error.
"""
import numpy as np
import pytest
import torch

from oracle import sample as os_

pytestmark = pytest.mark.gpu
SLACK = 2.0 ** -28
INF = float("inf")
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def ss():
    from speculative_decoding_verification_35_gb300 import specsample
    return specsample


def make(rows, V, kind, sigma=2.5, zipf=1.1, seed=0, pad=0, shift=0):
    """Rows of a model's logits, stride V + pad, the first `shift` elements into their memory."""
    g = torch.Generator("cuda").manual_seed(seed)
    x = torch.randn((rows, V), generator=g, device="cuda") * sigma - zipf * torch.arange(1, V + 1, device="cuda").log()
    return place(x.to(DT[kind]), pad, shift)


def place(x, pad=0, shift=0):
    rows, V = x.shape
    full = torch.full((rows * (V + pad) + shift + 8,), float("nan"), dtype=x.dtype, device="cuda")
    at = full[shift:shift + rows * (V + pad)].view(rows, V + pad)[:, :V]
    at.copy_(x)
    return at


def requests(rows, T=None, k=None, p=None, mp=None):
    def t(v, kind):
        if v is None:
            return None
        return torch.tensor(np.broadcast_to(np.asarray(v), (rows,)).copy(), dtype=kind, device="cuda")
    return t(T, torch.float32), t(k, torch.int32), t(p, torch.float32), t(mp, torch.float32)


def run(ss, x, f, u=None, out=None):
    """(tokens, logprobs, kept by sample, masked logits, kept by mask, status bits)."""
    rows = len(x)
    i32 = dict(dtype=torch.int32, device="cuda")
    u = torch.rand(rows, device="cuda", generator=torch.Generator("cuda").manual_seed(3)) if u is None else u
    tok, n1, n2 = torch.full((rows,), -7, **i32), torch.full((rows,), -7, **i32), torch.full((rows,), -7, **i32)
    lp = torch.full((rows,), 7.0, device="cuda")
    out = torch.full(x.shape, 5.0, dtype=x.dtype, device="cuda") if out is None else out
    f.status.zero_()
    assert f.sample(x, u, tok, lp, n1) == 0
    assert f.mask(x, out, n2) == 0
    torch.cuda.synchronize()
    return tok, lp, n1, out, n2, f.status_bits()


def check(ss, x, T=None, k=None, p=None, mp=None, u=None, out=None, request=None, seed=3):
    rows = len(x)
    n = rows if request is None else int(max(request)) + 1
    f = ss.Filter(*requests(n, T, k, p, mp), device="cuda",
                  request=None if request is None else torch.tensor(request, dtype=torch.int32, device="cuda"))
    if u is None:
        u = torch.rand(rows, device="cuda", generator=torch.Generator("cuda").manual_seed(seed))
    tok, lp, n1, y, n2, bits = run(ss, x, f, u, out)
    assert bits == 0
    l = x.double().cpu().numpy()
    y, tok, lp, n1, n2, u = (t.double().cpu().numpy() for t in (y, tok, lp, n1, n2, u))
    assert np.array_equal(n1, n2)

    def of(v, r, default):
        v = default if v is None else np.broadcast_to(np.asarray(v), (n,))[r if request is None else request[r]]
        return v if isinstance(v, (int, np.integer)) else float(np.float32(v))
    for r in range(rows):
        Tr, kr, pr, mr = of(T, r, 1.0), of(k, r, 0), of(p, r, 1.0), of(mp, r, 0.0)
        lo, hi = os_.counts(l[r], Tr, int(kr), pr, mr, SLACK)
        got = int(n1[r])
        assert lo <= got <= hi, (r, got, lo, hi)
        keep = os_.kept(l[r], got)
        assert np.array_equal(y[r], np.where(keep, l[r], -np.inf)), r
        a, b, logp = os_.draws(l[r], Tr, keep, float(u[r]), SLACK)
        t = int(tok[r])
        assert a <= t <= b and keep[t], (r, t, a, b)
        assert abs(lp[r] - logp[t]) <= 2.0 ** -24 * abs(logp[t]) + SLACK, (r, lp[r], logp[t])


SIZES = [1, 2, 3, 7, 8, 9, 31, 64, 100, 513, 1023, 1024, 4097, 32000, 50001, 128256, 152064, 200001, 262144]


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("V", SIZES)
def test_every_size(ss, V, kind):
    rows = 6
    x = make(rows, V, kind, seed=V, pad=V % 5, shift=V % 3)
    check(ss, x, T=[1.0, 0.7, 1.3, 1.0, 0.9, 0.0], k=[0, 50, 7, 0, 1, 3], p=[1.0, 1.0, 0.9, 0.8, 0.5, 0.9],
          mp=[0.0, 0.0, 0.0, 0.05, 0.0, 0.3])


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("kw", [dict(), dict(k=40), dict(p=0.9), dict(p=0.999), dict(mp=0.03), dict(T=0.0), dict(T=0.05), dict(T=40.0),
                                dict(T=1e30), dict(T=1e-30), dict(k=300, p=0.95), dict(k=5, p=0.3, mp=0.2, T=0.8), dict(p=0.0),
                                dict(p=-1.0), dict(p=1e-30), dict(mp=1.0), dict(mp=7.0), dict(mp=1e-30), dict(k=-5), dict(k=2 ** 31 - 1),
                                dict(k=1)])
def test_filters(ss, kind, kw):
    check(ss, make(9, 5003, kind, seed=11, pad=3), **kw)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 2, 5, 19, 40, 77, 160, 400])
def test_every_batch(ss, rows, kind):
    rng = np.random.default_rng(rows)
    check(ss, make(rows, 9001, kind, seed=rows, sigma=1.5), T=rng.choice([0.0, 0.6, 1.0, 1.4], rows), k=rng.choice([0, 3, 200], rows),
          p=rng.choice([1.0, 0.7, 0.95], rows), mp=rng.choice([0.0, 0.1], rows))


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("what", ["equal", "two", "zeros", "hidden", "one", "tiny", "huge", "low", "around", "ladder"])
def test_values(ss, kind, what):
    """Rows of few values, values outside the quick bins, hidden tokens, zeros of both signs."""
    V = 40000
    g = torch.Generator("cuda").manual_seed(5)
    x = torch.randn((8, V), generator=g, device="cuda")
    if what == "equal":
        x[:] = 3.25
    elif what == "two":
        x = (x > 1).float() * 2.0
    elif what == "zeros":
        x = torch.where(x > 0, 0.0, -0.0)
        x[:, ::1000] = 1.0
    elif what == "hidden":
        x[x < 1] = -INF
    elif what == "one":
        x[:] = -INF
        x[:, 12345] = -50.0
    elif what == "tiny":
        x = x * 1e-9
    elif what == "huge":
        x = x * 3000
    elif what == "low":
        x = x - 5000.0
    elif what == "around":  # some outside, none of which matters, and the crossing among the others
        x[:, 7] = 1e-20
        x[:, 9] = -1e30
    else:
        x = -0.01 * torch.arange(V, device="cuda", dtype=torch.float32).expand(8, V).contiguous()
    x = place(x.to(DT[kind]), 1, 1)
    check(ss, x, T=[1.0, 1.0, 2.0, 1.0, 0.0, 1.0, 300.0, 1.0], k=[0, 100, 0, 777, 5, 0, 0, 20001], p=[0.5, 1.0, 0.9, 0.31, 0.5, 1.0, 0.5, 0.7],
          mp=[0.0, 0.0, 0.0, 0.0, 0.0, 0.2, 0.0, 0.0])


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_uniforms_at_the_ends(ss, kind):
    x = make(6, 3001, kind, seed=2)
    x[:, 0] = -INF
    u = torch.tensor([0.0, 1.0 - 2.0 ** -24, 1e-38, 0.5, 1e-45, 2.0 ** -24], device="cuda")
    check(ss, x, u=u)
    check(ss, x, u=u, k=3)
    check(ss, x, u=u, p=0.6)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_shared_requests(ss, kind):
    x = make(12, 4000, kind, seed=8)
    check(ss, x, T=[0.5, 1.0, 2.0], k=[9, 0, 30], p=[1.0, 0.9, 0.8], request=[0, 0, 1, 2, 1, 1, 0, 2, 2, 2, 0, 1])


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("pad,shift", [(0, 0), (0, 1), (3, 2), (8, 5), (1, 0)])
def test_output_anywhere(ss, kind, pad, shift):
    x = make(5, 2050, kind, seed=4, pad=2, shift=3)
    out = place(torch.zeros_like(x), pad, shift)
    whole = out.as_strided((5 * (2050 + pad) + shift + 8,), (1,), 0)
    check(ss, x, k=30, p=0.9, out=out)
    rest = torch.ones_like(whole, dtype=torch.bool)
    rest.as_strided(out.shape, out.stride(), shift)[:] = False
    assert whole[rest].isnan().all()  # nothing beside the rows is written


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("V", [5, 3001, 128256])
def test_in_place(ss, V, kind):
    x = make(4, V, kind, seed=9, pad=1)
    f = ss.Filter(*requests(4, 0.9, 20, 0.9, None))
    want = torch.empty_like(x).contiguous()
    assert f.mask(x, want) == 0
    assert f.mask(x, x) == 0
    assert torch.equal(x, want)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_findings_fail_their_row_alone(ss, kind):
    from speculative_decoding_verification_35_gb300 import specverify as sv
    V = 6001
    clean = make(12, V, kind, seed=1)
    x = clean.clone()
    x[1, 5] = float("nan")
    x[2, V - 1] = INF
    x[3] = -INF
    x[11, 0] = -float("nan")
    T, k, p, mp = requests(12, 1.0, 20, 0.9, 0.01)
    T[4], T[5], T[6] = -1.0, INF, float("nan")
    p[7], mp[8] = float("nan"), float("nan")
    req = torch.arange(12, dtype=torch.int32, device="cuda")
    req[9] = 12
    u = torch.full((12,), 0.4, device="cuda")
    u[10] = 1.0
    f = ss.Filter(T, k, p, mp, req)
    tok, lp, n1, y, n2, bits = run(ss, x, f, u)
    assert bits == 1 << sv.SV_ERR_NONFINITE | 1 << sv.SV_ERR_EMPTY_ROW | 1 << sv.SV_ERR_INVALID_ARG
    assert tok[1:].tolist() == [-1] * 11 and tok[0] >= 0
    assert lp[1:].isnan().all() and lp[0].isfinite()
    assert n1[1:].tolist() == [-1] * 11
    assert n2[1:].tolist() == [-1] * 9 + [int(n2[10])] + [-1] and n2[10] > 0  # the uniform is none of the filter's
    same = [1, 2, 3, 4, 5, 6, 7, 8, 9, 11]
    view = torch.int16 if kind == "bf16" else torch.int32
    assert torch.equal(y[same].view(view), x[same].contiguous().view(view))
    one = run(ss, x[:1], ss.Filter(T[:1], k[:1], p[:1], mp[:1]), u[:1])
    assert one[5] == 0 and one[0][0] == tok[0] and torch.equal(one[3][0], y[0])


def test_a_finding_of_a_negative_uniform(ss):
    x = make(2, 100, "f32")
    f = ss.Filter(device="cuda")
    for bad in (-1e-9, float("nan"), 1.5):
        tok = run(ss, x, f, torch.tensor([bad, 0.5], device="cuda"))
        assert tok[0][0] == -1 and tok[0][1] >= 0 and tok[5] == 2


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_results_do_not_depend_on_the_batch(ss, kind):
    """A row alone and in a large batch: other cluster sizes, the same bits."""
    x = make(200, 30011, kind, seed=6)
    u = torch.rand(200, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    T, k, p, mp = requests(200, 0.8, None, 0.95, None)
    many = run(ss, x, ss.Filter(T, k, p, mp), u)
    for r in (0, 63, 199):
        one = run(ss, x[r:r + 1], ss.Filter(T[:1], None, p[:1], None), u[r:r + 1])
        for a, b in zip(one[:5], many[:5]):
            assert torch.equal(a[0], b[r])


def test_streams_and_graphs(ss):
    """Two calls at once on two streams, and a captured pair replayed on new inputs."""
    x = [make(30, 20001, "bf16", seed=s) for s in (1, 2)]
    u = torch.rand(30, device="cuda")
    fs = [ss.Filter(*requests(30, 1.0, kk, 0.9, None)) for kk in (50, 0)]
    want = [run(ss, x[i], fs[i], u) for i in (0, 1)]
    got = []
    torch.cuda.synchronize()
    for i in (0, 1):
        st = torch.cuda.Stream()
        tok, out = torch.empty(30, dtype=torch.int32, device="cuda"), torch.empty_like(x[i])
        torch.cuda.synchronize()
        for _ in range(5):
            assert fs[i].sample(x[i], u, tok, stream=st) == 0
            assert fs[i].mask(x[i], out, stream=st) == 0
        got.append((tok, out))
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert torch.equal(w[0], g[0]) and torch.equal(w[3], g[1])
    held, tok, out = x[0].clone(), torch.empty(30, dtype=torch.int32, device="cuda"), torch.empty_like(x[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        assert fs[0].sample(held, u, tok) == 0
        assert fs[0].mask(held, out) == 0
    for i in (0, 1, 0):
        held.copy_(x[i])
        graph.replay()
        w = run(ss, x[i], fs[0], u)
        assert torch.equal(w[0], tok) and torch.equal(w[3], out)


def test_no_rows(ss):
    x = torch.empty((0, 50), device="cuda")
    f = ss.Filter(device="cuda")
    assert f.mask(x, x) == 0
    assert f.sample(x, torch.empty(0, device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda")) == 0


def test_draws_follow_the_distribution(ss):
    """Many uniforms on one row: the counts of each kept token (a grid of uniforms: off by one at most, and by the
    roundings at either border)."""
    n, V = 4096, 600
    x = make(1, V, "bf16", sigma=1.0, seed=3).expand(n, V).contiguous()
    u = (torch.arange(n, device="cuda") + 0.5) / n
    tok = run(ss, x, ss.Filter(*requests(n, 0.9, 100, 0.95, None)), u)[0].cpu().numpy()
    l = x[0].double().cpu().numpy()
    T, p = float(np.float32(0.9)), float(np.float32(0.95))
    keep = os_.kept(l, os_.counts(l, T, 100, p)[0])
    want = np.exp(os_.draws(l, T, keep, 0.5)[2]) * n
    assert (np.abs(np.bincount(tok, minlength=V) - want) <= 1.0 + 2 * SLACK * n).all()


@pytest.mark.parametrize("drafts", [True, False])
def test_a_verify_step_on_filtered_rows(ss, drafts):
    """Drafts drawn from filtered rows, both rows filtered, verified: what the verify oracle says of the same rows."""
    import oracle
    from speculative_decoding_verification_35_gb300 import specverify as sv
    B, g, V, T = 8, 4, 8000, 0.7
    target, draft = make(B * (g + 1), V, "bf16", seed=21), make(B * g, V, "bf16", seed=21)
    draft.copy_((target.view(B, g + 1, V)[:, :g].float() + 0.5 * torch.randn((B, g, V), device="cuda",
                 generator=torch.Generator("cuda").manual_seed(4))).to(torch.bfloat16).view(B * g, V))
    i32 = dict(dtype=torch.int32, device="cuda")
    per = requests(B, T, [0, 20, 50, 0, 7, 100, 0, 3], [0.9, 1.0, 0.8, 0.95, 1.0, 0.7, 0.5, 1.0], 0.01)
    tf = ss.Filter(*per, request=torch.arange(B, **i32).repeat_interleave(g + 1))
    df = ss.Filter(*per, request=torch.arange(B, **i32).repeat_interleave(g))
    tokens = torch.empty(B * g, **i32)
    u = torch.rand(B * g, device="cuda", generator=torch.Generator("cuda").manual_seed(7))
    assert df.sample(draft, u, tokens) == 0
    assert df.mask(draft, draft) == 0 and tf.mask(target, target) == 0
    assert bool((draft.gather(1, tokens.long()[:, None]) > -INF).all())  # every draft is a token of its filtered row
    offs, gam = torch.arange(B + 1, **i32) * g, torch.full((B,), g, **i32)
    call = sv.Call(B, V, g, B * (g + 1), B * g)
    assert call.run(target, draft if drafts else None, tokens, offs, gam, T, 99, 5) == 0
    torch.cuda.synchronize()
    assert call.status_bits() == 0 and tf.status_bits() == 0 and df.status_bits() == 0
    def bits(t):
        return t.view(torch.int16).cpu().numpy().view(np.uint16)
    ref = oracle.verify(bits(target), bits(draft) if drafts else None, tokens.cpu().numpy(), offs.cpu().numpy(), gam.cpu().numpy(), V,
                        T, 99, 5)
    assert np.array_equal(call.out_n.cpu().numpy(), ref.num_accepted)
    got = call.out_tokens.cpu().numpy()
    assert np.array_equal(got, ref.tokens)
    rows = np.flatnonzero(got >= 0)  # an emitted token is one that the filtered target allows
    assert bool((target[torch.tensor(rows, device="cuda")].gather(1, torch.tensor(got[rows], device="cuda").long()[:, None]) > -INF).all())


# Rows too many to be held in shared memory at once are read where they lie, one CTA an SM.
MANY = {"bf16": (150, 128256), "f32": (60, 129281)}


def many(kind, seed, pad=0, shift=0):
    rows, V = MANY[kind]
    x = make(rows, V, kind, seed=seed, pad=pad, shift=shift)
    x[3] = 1.5                                                # all alike
    x[4, ::2] = -INF                                          # hidden tokens
    x[5, :] = -INF
    x[5, V - 1] = 0.0                                         # one is left, the last
    x[6] = (x[6].float() * 3e4).to(x.dtype)                   # outside the quick bins
    x[7] = (x[7].float() * 1e-12).to(x.dtype)
    kw = dict(T=[1.0, 0.7, 1.0, 1.3, 0.9, 1.0, 0.0], k=[0, 50, 0, 5000, 0, 1, 1000, 0, 0], p=[0.9, 1.0, 1.0, 0.95, 0.999],
              mp=[0.0, 0.0, 0.02, 0.0])
    return x, {n: np.resize(np.asarray(v), rows) for n, v in kw.items()}


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("pad,shift", [(0, 0), (3, 1)])
def test_rows_read_where_they_lie(ss, kind, pad, shift):
    x, kw = many(kind, 21, pad, shift)
    check(ss, x, **kw)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("pad,shift", [(0, 0), (5, 3)])
def test_rows_read_where_they_lie_are_as_alone(ss, kind, pad, shift):
    """Tokens, counts and masked rows (elsewhere, and in place) are those of the same rows a few at a time, which are held."""
    x, kw = many(kind, 22, 1, 2)
    rows, V = x.shape
    u = torch.rand(rows, device="cuda", generator=torch.Generator("cuda").manual_seed(8))
    f = ss.Filter(*requests(rows, **kw), device="cuda")
    tok, lp, n1, y, n2, bits = run(ss, x, f, u, place(torch.zeros_like(x), pad, shift))
    assert bits == 0
    for a in range(0, rows, 10):
        g = ss.Filter(*requests(len(u[a:a + 10]), **{n: v[a:a + 10] for n, v in kw.items()}), device="cuda")
        got = run(ss, x[a:a + 10], g, u[a:a + 10])
        for all_, few in zip((tok, lp, n1, y, n2), got):
            assert torch.equal(all_[a:a + 10], few), a
    assert f.mask(x, x, n2) == 0
    torch.cuda.synchronize()
    assert torch.equal(x, y) and torch.equal(n1, n2)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_findings_where_rows_are_read_where_they_lie(ss, kind):
    x, kw = many(kind, 23)
    want = run(ss, x, ss.Filter(*requests(len(x), **kw), device="cuda"))
    bad = [0, 11, 40]
    y = x.clone()
    y[0, 5], y[11, -1], y[40] = float("nan"), INF, -INF
    tok, lp, n1, out, n2, bits = run(ss, y, ss.Filter(*requests(len(x), **kw), device="cuda"))
    assert bits != 0
    good = [r for r in range(len(x)) if r not in bad]
    for a, b in zip((tok, lp, n1, out, n2), want):
        assert torch.equal(a[good], b[good])


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("V", [7, 5003])
def test_the_largest_temperature(ss, kind, V):
    """A logit that lies further below the largest than float reaches has no weight up to T = 1e36; above, it would have one
    (2^-8.7 at 1e38), and the row is refused."""
    from speculative_decoding_verification_35_gb300 import specverify as sv
    x = torch.full((4, V), -3e38, device="cuda")
    x[:, 1::3] = 3e38
    x = x.to(DT[kind])
    u = torch.full((4,), 0.999, device="cuda")
    T = float(np.float32(1e36))
    check(ss, x, T=T, u=u)
    check(ss, x, T=T, p=0.9, u=u)
    for worse in (2e36, 1e38, 3.4e38):
        tok, lp, n1, y, n2, bits = run(ss, x, ss.Filter(*requests(4, worse), device="cuda"), u)
        assert bits == 1 << sv.SV_ERR_INVALID_ARG
        assert tok.tolist() == [-1] * 4 and n1.tolist() == n2.tolist() == [-1] * 4 and torch.equal(y, x)
