"""rl_sample on the GPU against the definition in 64 bits.

Bounds.  A kernel's weight e is good to 2^-30 of itself and is kept in multiples of 2^-46 of the largest, so a sum of
weights is off by at most 2^-30 of itself + V 2^-46 (V up to 2^17).  Where a border of the definition (a running sum against its
target) is nearer than 2^-28 of the total, either side may be right, and the row is not compared; otherwise the token has
to be the definition's.  A distance of exactly 0 is that of equal logits (weights of 1, sums and targets that are exact on both
sides), and is compared.  The log probability is a sum of two f32 results: four half steps of each part."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = 2.0 ** -24
NEAR = 2.0 ** -28
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def L():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from quantized_moe_expert_rl_gb300 import _lib, build
    build.build()
    return _lib


def define(x, u, heat=1.0, k=0, p=1.0, m=0.0):
    """(token, log probability, error allowed in it, distance of the nearest border) of one row."""
    x = x.double().cpu()
    V = x.numel()
    if bool(torch.isnan(x).any()) or float(x.max()) == math.inf or float(x.max()) == -math.inf:
        return -1, math.nan, 0.0, 1.0
    top = x.max()
    if not heat > 0 or k == 1:
        return int((x == top).nonzero()[0, 0]), 0.0, 0.0, 1.0
    order = torch.argsort(-x, stable=True)
    z = (x[order] - top) / heat
    if 0 < k < V:
        order, z = order[:k], z[:k]
    e = z.exp()
    near = 1.0
    if p < 1:
        cum = e.cumsum(0)
        share = max(p, 0.0) * cum[-1]
        n = max(1, int((cum - e < share).sum()))
        # the sums on both sides of the last kept token
        near = min(near, float((cum[n - 1] - share).abs() / cum[-1]), float((share - (cum[n - 1] - e[n - 1])).abs() / cum[-1]) if n > 1 else 1.0)
        order, z, e = order[:n], z[:n], e[:n]
    if m > 0:
        n = max(1, int((z >= math.log(min(m, 1.0))).sum()))
        order, z, e = order[:n], z[:n], e[:n]
    ids, at = order.sort()
    e, z = e[at], z[at]
    cum = e.cumsum(0)
    r = min(max(0.0 if math.isnan(u) else u, 0.0), 1.0) * float(cum[-1])
    j = min(int((cum <= r).sum()), int((e > 0).nonzero()[-1, 0]))
    if u < 1:
        near = min(near, float((cum[j] - r).abs() / cum[-1]), float((r - (cum[j] - e[j])).abs() / cum[-1]) if r > 0 else 1.0)
    lp = float(z[j]) - math.log(float(cum[-1]))
    return int(ids[j]), lp, 4 * U * (abs(float(z[j])) + abs(math.log(float(cum[-1])))) + 2.0 ** -29, near


def check(L, x, u, heat=None, k=None, p=None, m=None, least=0.9):
    T, V = x.shape
    row = lambda v, t, dt: v if v is None or torch.is_tensor(v) else torch.full((T,), v, dtype=dt)  # noqa: E731
    heat, k, p, m = row(heat, T, torch.float32), row(k, T, torch.int32), row(p, T, torch.float32), row(m, T, torch.float32)
    dev = lambda v: None if v is None else v.cuda()  # noqa: E731
    ids = torch.full((T,), -7, dtype=torch.int32, device="cuda")
    lp = torch.full((T,), 7.0, device="cuda")
    L.rl_sample(x, T, V, dev(u), ids, temperature=dev(heat), top_k=dev(k), top_p=dev(p), min_p=dev(m), logprob=lp)
    alone = torch.full_like(ids, -7)
    L.rl_sample(x, T, V, dev(u), alone, temperature=dev(heat), top_k=dev(k), top_p=dev(p), min_p=dev(m))
    assert torch.equal(ids, alone)
    compared = 0
    for t in range(T):
        val = lambda v, d: d if v is None else v[t].item()  # noqa: E731
        want, wlp, err, near = define(x[t], float(u[t]), val(heat, 1.0), val(k, 0), val(p, 1.0), val(m, 0.0))
        if 0 < near < NEAR:
            continue
        compared += 1
        assert int(ids[t]) == want, (t, int(ids[t]), want, near)
        got = float(lp[t])
        assert (math.isnan(wlp) and math.isnan(got)) or abs(got - wlp) <= err, (t, got, wlp)
    assert compared >= least * T
    return ids


def logits(kind, T, V, seed, dt=torch.float32):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, V, generator=g)
    if kind == "peaked":
        x = 2 * x - 4
        x.scatter_(1, torch.randint(0, V, (T, min(V, 12)), generator=g), 9 + 3 * torch.randn(T, min(V, 12), generator=g))
    elif kind == "flat":
        x = torch.full((T, V), 1.25)
    elif kind == "steps":
        x = torch.randint(0, 5, (T, V), generator=g).float()
    elif kind == "masked":
        x = torch.where(torch.rand(T, V, generator=g) < 0.97, torch.full_like(x, -math.inf), 3 * x)
        x[:, V // 2] = 0.5
    elif kind == "lowest":
        x = torch.where(torch.rand(T, V, generator=g) < 0.5, torch.full_like(x, torch.finfo(dt).min), x)
        x[:, V // 3] = 0.5
    return x.to(dt).cuda(), torch.rand(T, generator=g)


KINDS = ["peaked", "broad", "flat", "steps", "masked", "lowest"]


@pytest.mark.parametrize("V", [1, 2, 31, 1000, 2049, 4097, 9001, 32000, 100003, 131072])
@pytest.mark.parametrize("kind", KINDS)
def test_sample_settings(L, kind, V):
    T = 6
    for i, (heat, k, p, m) in enumerate([(None, None, None, None), (0.7, 50, 0.9, None), (1.3, None, 0.95, 0.02),
                                         (None, 3000, None, None), (1.0, 300, 0.5, None), (2.0, 5000, 0.99, 0.001),
                                         (None, None, 0.3, None), (0.9, 20, None, 0.1), (0.0, None, 0.9, None), (1.0, 1, None, None),
                                         (0.5, 2, 0.6, None)]):
        dt = list(TYPES.values())[i % 3]
        x, u = logits(kind, T, V, 17 * V + i, dt)
        check(L, x, u, heat, k, p, m)


@pytest.mark.parametrize("T,V,dt", [(1, 131072, "f32"), (300, 20011, "bf16"), (70, 131072, "f32"), (3, 262144, "f32"),
                                    (2, 500001, "f32"), (2, 900001, "f16"), (2, 1500000, "bf16")])
@pytest.mark.parametrize("kind", ["peaked", "broad", "steps"])
def test_sample_sizes(L, kind, T, V, dt):
    """Rows over one to eight CTAs, in shared memory and beyond it, with settings of their own."""
    x, u = logits(kind, T, V, T + V, TYPES[dt])
    g = torch.Generator().manual_seed(T)
    pick = lambda v: torch.tensor(v)[torch.randint(0, len(v), (T,), generator=g)]  # noqa: E731
    check(L, x, u, pick([0.0, 0.5, 1.0, 1.5]), pick([0, 1, 40, 2000, V // 2]).int(), pick([1.0, 0.4, 0.9, 0.99]), pick([0.0, 0.05]))
    check(L, x, u)


def test_sample_borders(L):
    """u at both ends and outside, settings at and beyond their ends, equal logits in index order."""
    nan, inf = math.nan, math.inf
    x, _ = logits("steps", 8, 5000, 3)
    u = torch.tensor([0.0, 1.0, -1.0, 2.0, nan, 1 - 2.0 ** -24, 0.5, 2.0 ** -24])
    check(L, x, u, least=1.0)
    check(L, x, u, 1.0, torch.tensor([-1, 0, 4999, 5000, 5001, 2 ** 31 - 1, -2 ** 31, 7], dtype=torch.int32), least=0.8)
    check(L, x, u, p=torch.tensor([0.0, -1.0, 1.0, 1.5, nan, inf, -inf, 1e-30]), least=0.8)
    check(L, x, u, m=torch.tensor([0.0, -1.0, 1.0, 1.5, nan, inf, -inf, 1e-30]), least=0.8)
    check(L, x, u, heat=torch.tensor([0.0, -1.0, nan, -inf, 1e-20, 1e20, inf, 1e-3]), least=0.8)
    x, u = logits("flat", 4, 70001, 1)
    x[:, 5] = -0.0
    x[:, 6] = 0.0
    check(L, x * 0, u, k=30000)
    check(L, x, u, p=0.37)


def test_sample_broken_rows(L):
    """NaN, infinities, rows without a distribution; the rows beside them are as alone."""
    x, u = logits("broad", 9, 40000, 5)
    sole = x.clone()
    x[1, 77] = math.nan
    x[3, 39999] = math.inf
    x[5] = -math.inf
    x[6, :-1] = -math.inf
    x[7] = math.nan
    for kw in ({}, {"k": 50, "p": 0.9}, {"heat": 0.0}, {"p": 0.99}, {"k": 9000}):
        ids = check(L, x, u, **kw)
        assert [int(i) for i in ids[[1, 3, 5, 7]]] == [-1] * 4 and int(ids[6]) == 39999
        good = check(L, sole, u, **kw)
        assert torch.equal(ids[[0, 2, 4, 8]], good[[0, 2, 4, 8]])


def test_sample_magnitudes(L):
    """Logits at the ends of f32 and f16, subnormal differences, tiny and huge temperatures."""
    g = torch.Generator().manual_seed(2)
    x = torch.randn(6, 3000, generator=g)
    u = torch.rand(6, generator=g)
    check(L, (x * 8e37).cuda(), u)
    check(L, (x * 8e37).cuda(), u, heat=1e37, p=0.9)
    check(L, (x * 1e-40).cuda(), u, k=100)
    check(L, (x * 1e-40).cuda(), u, heat=1e-22)
    check(L, (x * 1e-3 + 1000).cuda(), u, heat=1e-3, p=0.8)
    check(L, (x * 15000).half().cuda(), u, heat=500.0, k=200, p=0.95)
    check(L, (x * 1e-7).half().cuda(), u, heat=1e-7, p=0.7)


def test_sample_unaligned(L):
    """Rows that start anywhere, and more of them than fit the GPU at once."""
    for dt in TYPES.values():
        flat, _ = logits("peaked", 1, 3 * 10007 + 5, 9, dt)
        for skip in (0, 1, 3, 5):
            check(L, flat[0, skip:skip + 3 * 10007].view(3, 10007), torch.rand(3, generator=torch.Generator().manual_seed(skip)), 1.0, 30, 0.9)
    x, u = logits("peaked", 700, 1500, 4)
    check(L, x, u, 1.0, 30, 0.9)


def test_sample_graph_and_stream(L):
    """A captured call draws anew from the numbers in its buffer; another stream than the current one."""
    x, u = logits("broad", 20, 50000, 8)
    u = u.cuda()
    ids, lp = torch.zeros(20, dtype=torch.int32, device="cuda"), torch.zeros(20, device="cuda")
    p = torch.full((20,), 0.9, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    L.rl_sample(x, 20, 50000, u, ids, top_p=p, logprob=lp, stream=s)
    s.synchronize()
    first = ids.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        L.rl_sample(x, 20, 50000, u, ids, top_p=p, logprob=lp)
    u.copy_(1 - u)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    other, again = ids.clone(), torch.zeros_like(ids)
    assert not torch.equal(first, other)
    L.rl_sample(x, 20, 50000, u, again, top_p=p)
    assert torch.equal(again, other)
    u.copy_(1 - u)
    g.replay()
    # 1 - (1 - u) rounds u: the token is the same but where a border lies between
    assert int((ids != first).sum()) <= 2


def test_sample_follows_the_distribution(L):
    """100 000 draws from one row, by their counts: chi-square below its mean plus six standard deviations."""
    V, N = 40, 100_000
    g = torch.Generator().manual_seed(6)
    x = (1.5 * torch.randn(1, V, generator=g)).cuda()
    rows = x.expand(N, V).contiguous()
    ids = torch.zeros(N, dtype=torch.int32, device="cuda")
    L.rl_sample(rows, N, V, torch.rand(N, generator=g).cuda(), ids)
    want = torch.softmax(x[0].double(), 0) * N
    got = torch.bincount(ids.long(), minlength=V).double()
    chi = float(((got - want) ** 2 / want).sum())
    assert chi < (V - 1) + 6 * math.sqrt(2 * (V - 1))


def near_ties(m, T, V, seed):
    """Rows of m and the 64 f32 values below it, in any order, m at least once."""
    steps = [torch.tensor(m)]
    for _ in range(64):
        steps.append(torch.nextafter(steps[-1], torch.tensor(-math.inf)))
    g = torch.Generator().manual_seed(seed)
    x = torch.stack(steps)[torch.randint(0, 65, (T, V), generator=g)]
    x[:, V // 3] = m
    return x.cuda(), torch.rand(T, generator=g)


@pytest.mark.parametrize("m", [1.0, 5.0, 20.0, 1000.0, 1e8, 1e-20, -20.0, 3e38])
def test_sample_near_ties(L, m):
    """Logits a few f32 steps apart and temperatures beside those steps: from all weights alike to the largest's alone, with the last
    logit that has a weight anywhere between."""
    heat = torch.cat([torch.logspace(-8, 0, 33), (abs(m) * torch.logspace(-9, -4, 61, dtype=torch.float64)).float()])
    for i, kw in enumerate(({}, {"p": 0.9}, {"m": 0.01}, {"k": 400}, {"k": 300, "p": 0.8}, {"p": 0.99, "m": 1e-6})):
        x, u = near_ties(m, len(heat), 1000, 31 * i + 7)
        check(L, x, u, heat=heat, **kw)


def test_sample_huge_temperatures(L):
    """Logits of both signs up to the largest f32, whose differences leave the type, at temperatures that keep them all."""
    top = torch.finfo(torch.float32).max
    g = torch.Generator().manual_seed(12)
    heat = torch.tensor([1e35, 5e36, 1.07e37, 3e37, 1e38, top, math.inf, 2e38])
    T, V = len(heat), 3000
    u = torch.rand(T, generator=g)
    x = (2 * torch.rand(T, V, generator=g) - 1) * top
    x[:, 17], x[:, 2900] = top, -top
    big = x.bfloat16()
    big[torch.isinf(big)] = 1e38
    for kw in ({}, {"p": 0.9}, {"p": 0.3}, {"k": 100}, {"k": 2500, "p": 0.7}, {"k": 2500}, {"m": 0.2}, {"p": 0.95, "m": 0.05}):
        for rows in (x.cuda(), big.cuda()):
            ids = check(L, rows, u, heat=heat.clamp(max=top), **kw)  # (an infinite temperature counts as the largest f32)
            out = torch.full((T,), -7, dtype=torch.int32, device="cuda")
            k, p, m = (None if n not in kw else torch.full((T,), kw[n], dtype=dt, device="cuda")
                       for n, dt in (("k", torch.int32), ("p", torch.float32), ("m", torch.float32)))
            L.rl_sample(rows, T, V, u.cuda(), out, temperature=heat.cuda(), top_k=k, top_p=p, min_p=m)
            assert torch.equal(out, ids)
    x, u = logits("broad", T, 5000, 3)  # differences that such temperatures do not see
    check(L, x, u, heat=heat, p=0.6)


@pytest.mark.parametrize("T,V,dt", [(200, 40001, "f32"), (170, 70001, "bf16")])
def test_sample_many_long_rows(L, T, V, dt):
    """More rows than SMs, each streamed by two CTAs: settings of their own, flat rows with top-p, many kept tokens."""
    g = torch.Generator().manual_seed(V)
    pick = lambda v: torch.tensor(v)[torch.randint(0, len(v), (T,), generator=g)]  # noqa: E731
    for kind in ("peaked", "broad", "steps"):
        x, u = logits(kind, T, V, T + V, TYPES[dt])
        check(L, x, u, pick([0.0, 0.5, 1.0, 1.5]), pick([0, 1, 40, 5000, V // 2]).int(), pick([1.0, 0.4, 0.95]), pick([0.0, 0.05]))
    x, u = logits("flat", T, V, 5, TYPES[dt])
    check(L, x, u, p=0.95)
    x, u = logits("broad", T, V, 6, TYPES[dt])
    check(L, x, u, p=0.95)
