"""The operators of a step of a few tokens on the GPU, each against a plain computation in 64 bits.

Bounds.  u = 2^-24 is half a step of f32.  A sum of n positive f32 terms is off by at most (n - 1) u
of itself, a signed one by (n - 1) u of the sum of magnitudes; half a step of a narrower result
type is added where the result is rounded (eps / 2 relative)."""
import math
from dataclasses import replace

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import oracle  # noqa: E402
import synth  # noqa: E402
from tests._gpu_common import REL_F32, OracleSide, check_route, rel_l2, u64  # noqa: E402

U = 2.0 ** -24
F8 = torch.float8_e4m3fn
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
NO_EARLY_OUT = 0x7FFFFFFF


@pytest.fixture(scope="module")
def L():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from quantized_moe_expert_rl_gb300 import _lib, build
    build.build()
    return _lib


def randn(*shape, seed=0, dtype=torch.float32):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


# ---- rl_add_rmsnorm -----------------------------------------------------------------------
def norm_ref(x, res, gain, eps, dt):
    s = x if res is None else (x.float() + res.float()).to(dt)
    v = s.double()
    v = v / (v.square().mean(1, keepdim=True) + eps).sqrt()
    return s, v if gain is None else v * gain.double()


def check_norm(L, x, res, gain, eps, group, inplace=False):
    T, H = x.shape
    dt = x.dtype
    s, v = norm_ref(x, res, gain, eps, dt)
    x_in = x.clone()
    x_out = x_in if inplace else torch.full_like(x, 7)
    xn = torch.full_like(x, 7)
    q = torch.zeros(T, H, dtype=F8, device="cuda")
    scale = torch.full((T, H // group), 7.0, device="cuda")
    L.rl_add_rmsnorm(x_in, T, H, eps, res=res, gain=gain, x_out=x_out, xn=xn, q=q, scale=scale, group=group)
    torch.cuda.synchronize()
    assert torch.equal(x_out, s)
    # the sum of squares: 16 terms per thread, 5 shuffles, at most 32 warps; half of that for the
    # root, then the root, the division and two products
    f32 = ((16 + 5 + 32) / 2 + 6) * U
    half = 0 if dt == torch.float32 else torch.finfo(dt).eps / 2
    tiny = float(torch.finfo(dt).smallest_normal) * torch.finfo(dt).eps
    assert torch.all((xn.double() - v).abs() <= v.abs() * (half + f32) * (1 + 1e-3) + tiny)
    groups = v.view(T, H // group, group)
    top = groups.abs().amax(2)
    assert torch.all((scale.double() - top / 448).abs() <= top / 448 * (f32 + 2 * U) + 1e-45)
    # half a step of e4m3: 2^-4 relative, 2^-10 (of the scale) below its smallest normal
    back = q.double().view(T, H // group, group) * scale.double()[..., None]
    assert torch.all((back - groups).abs() <= groups.abs() * (2.0 ** -4 + 2 * f32) + 2.0 ** -10 * scale.double()[..., None] * 1.001)
    assert torch.all(back[top == 0] == 0)
    # each output alone gives the same bits
    for k, full in (("x_out", x_out), ("xn", xn)):
        out = torch.full_like(x, 7)
        L.rl_add_rmsnorm(x, T, H, eps, res=res, gain=gain, **{k: out})
        assert torch.equal(out, full)
    q2, s2 = torch.zeros_like(q), torch.zeros_like(scale)
    L.rl_add_rmsnorm(x, T, H, eps, res=res, gain=gain, q=q2, scale=s2, group=group)
    assert torch.equal(q2.view(torch.uint8), q.view(torch.uint8)) and torch.equal(s2, scale)


@pytest.mark.parametrize("T,H,group", [(1, 128, 32), (3, 256, 64), (5, 2048, 128), (2, 8192, 128), (7, 640, 32),
                                       (2, 16384, 64), (301, 384, 128), (33, 8320, 64)])
@pytest.mark.parametrize("dt", list(TYPES))
def test_add_rmsnorm(L, T, H, group, dt):
    x, r = randn(T, H, seed=T, dtype=TYPES[dt]), randn(T, H, seed=H, dtype=TYPES[dt])
    g = 1 + 0.3 * randn(H, seed=5)
    check_norm(L, x, r, g, 1e-6, group)
    check_norm(L, x, None, None, 0.0, group)
    check_norm(L, x, r, None, 1e-6, group, inplace=True)


def test_add_rmsnorm_magnitudes(L):
    """Zero rows, squares beyond f32 in both directions, a row of one spike."""
    x = randn(6, 512, seed=2)
    x[0] = 0
    x[1] *= 1e25
    x[2] *= 1e-25
    x[3] = 0
    x[3, 77] = -3.0
    x[4, :128] = 0
    check_norm(L, x, None, None, 1e-6, 128)
    check_norm(L, x[1:].contiguous(), None, None, 0.0, 32)
    check_norm(L, x[4:].contiguous() * 1e-37, None, None, 1e-6, 64)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("H", [128, 2048, 16384])
def test_add_rmsnorm_below_the_normal_range(L, dt, H):
    """Rows whose factor 1 / RMS leaves the f32 range (RMS below 2.9e-39) are of order 1 all the same, their
    zeros stay zeros, and the rows beside them keep their bits."""
    g = torch.Generator().manual_seed(H)
    size = torch.tensor([1e-40, 2e-39, 4e-39, 1.0, 1e-38, 1e-30, 3e-39], dtype=torch.float64)[:, None]
    x = torch.randn(7, H, generator=g, dtype=torch.float64) * size
    x[0, ::3] = 0
    x = x.to(TYPES[dt]).cuda()
    assert torch.all(x[1:].double().abs().amax(1) > 0)
    gain = 1 + 0.3 * randn(H, seed=5)
    check_norm(L, x, None, None, 0.0, 32)
    check_norm(L, x, None, gain, 0.0, 128)
    one = torch.zeros_like(x)           # a single smallest value in a row
    one[:, 5] = float(torch.finfo(TYPES[dt]).smallest_normal) * torch.finfo(TYPES[dt]).eps
    check_norm(L, one, None, None, 0.0, 64)
    plain, beside = torch.empty_like(x[3:4]), torch.empty_like(x)
    L.rl_add_rmsnorm(x[3:4], 1, H, 0.0, xn=plain)
    L.rl_add_rmsnorm(x, 7, H, 0.0, xn=beside)
    assert torch.equal(plain[0], beside[3])


def test_add_rmsnorm_without_eight_bits_takes_any_multiple_of_8(L):
    for H in (8, 24, 1000, 2056):
        x = randn(3, H, seed=H)
        xn = torch.empty_like(x)
        L.rl_add_rmsnorm(x, 3, H, 1e-6, xn=xn)
        _, v = norm_ref(x, None, None, 1e-6, x.dtype)
        assert torch.all((xn.double() - v).abs() <= v.abs() * 40 * U)


def test_add_rmsnorm_non_finite_stays_in_its_row(L):
    x = randn(4, 256, seed=9)
    x[1, 40], x[2, 200] = math.inf, math.nan
    xn, q, s = torch.empty_like(x), torch.zeros(4, 256, dtype=F8, device="cuda"), torch.zeros(4, 8, device="cuda")
    L.rl_add_rmsnorm(x, 4, 256, 1e-6, xn=xn, q=q, scale=s, group=32)
    _, v = norm_ref(x, None, None, 1e-6, x.dtype)
    assert torch.equal(xn.isnan(), v.isnan())
    assert s[1].isnan().tolist() == [i == 1 for i in range(8)] and s[2].isnan().all()
    assert torch.all(s[1][[0, 2, 3, 4, 5, 6, 7]] == 0) and torch.all(q.float()[1:3] == 0)
    assert s[0].isfinite().all() and s[3].isfinite().all()


def test_add_rmsnorm_in_place_of_either_input(L):
    x, r = randn(9, 1024, seed=1, dtype=torch.bfloat16), randn(9, 1024, seed=2, dtype=torch.bfloat16)
    xn, xo = torch.empty_like(x), torch.empty_like(x)
    L.rl_add_rmsnorm(x, 9, 1024, 1e-6, res=r, x_out=xo, xn=xn)
    a, b = x.clone(), r.clone()
    L.rl_add_rmsnorm(a, 9, 1024, 1e-6, res=b, x_out=a, xn=b)
    assert torch.equal(a, xo) and torch.equal(b, xn)
    a, b = x.clone(), r.clone()
    L.rl_add_rmsnorm(a, 9, 1024, 1e-6, res=b, x_out=b, xn=a)
    assert torch.equal(b, xo) and torch.equal(a, xn)


# ---- rl_q4_matvec -------------------------------------------------------------------------
def q4_case(N, K, T, group, xt, seed=0):
    g = torch.Generator().manual_seed(seed)
    w = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8).cuda()
    ws = (0.001 + 0.01 * torch.rand(N, K // group, generator=g)).half().cuda()
    x = torch.randn(T, K, generator=g).cuda()
    x[:, :: 97] *= 50
    xs = None
    if xt == "f8":
        xs = x.view(T, K // group, group).abs().amax(2) / 448
        x = (x.view(T, K // group, group) / xs[:, :, None]).view(T, K).to(F8)
    else:
        x = x.to(TYPES[xt])
    return w, ws, x, xs


def q4_ref(w, ws, x, xs, group):
    """(y, sum of magnitudes, error of the activations' representation) in 64 bits."""
    N, K2 = w.shape
    T, K = x.shape
    q = torch.stack((w & 15, w >> 4), 2).view(N, 2 * K2).double()
    s = ws.double().repeat_interleave(group, 1)
    v = x.float().double()
    if xs is not None:
        v = v * xs.double().repeat_interleave(group, 1)
    top = v.view(T, K // group, group).abs().amax(2).repeat_interleave(group, 1)
    return v @ ((q - 8) * s).t(), v.abs() @ ((q + 8) * s).t(), top @ (8 * s).t()


def check_q4(y, ref, mag, rep, K, group, xt):
    # sums: group / 16 MMAs in a row of 16 products each (counted as 17 additions, truncated: 2 u
    # each), the offset's sum (8 + 4 shuffles), then 3 roundings per group over all groups of a row
    n = 2 * 17 * (group / 16) + 12 + 3 * (K // group) + 8
    half = torch.finfo(y.dtype).eps / 2 if y.dtype != torch.float32 else 0
    # f32 rows are held to 22 bits of each value, and to 2^-38 of the group's largest
    bound = mag * n * U + (mag * 2.0 ** -22 + rep * 2.0 ** -38 if xt == "f32" else rep * 2.0 ** -38) + ref.abs() * half + 1e-30
    err = (y.double() - ref).abs()
    assert torch.all(err <= bound), float((err / bound).max())
    if y.dtype == torch.float32:
        assert rel_l2(y.cpu().numpy(), ref.cpu().numpy()) <= REL_F32


@pytest.mark.parametrize("N,K,T,group", [(1, 128, 1, 128), (7, 32, 2, 32), (16, 256, 8, 64), (513, 2048, 1, 128),
                                         (100, 2048, 9, 32), (31, 384, 17, 64), (64, 8192, 3, 128), (2048, 512, 5, 64),
                                         (33, 4096, 33, 32), (40000, 256, 32, 64), (39000, 128, 40, 128), (17, 96, 70, 32)])
@pytest.mark.parametrize("xt", ["f8", "f32", "f16", "bf16"])
def test_q4_matvec(L, N, K, T, group, xt):
    w, ws, x, xs = q4_case(N, K, T, group, xt, seed=N)
    ref, mag, rep = q4_ref(w, ws, x, xs, group)
    guard = torch.full((T * N + 64,), 3.0, device="cuda")
    y = guard[:T * N].view(T, N)
    L.rl_q4_matvec(w, ws, x, y, T, N, K, group, x_scale=xs)
    check_q4(y, ref, mag, rep, K, group, xt)
    assert torch.all(guard[T * N:] == 3.0)
    first = y.clone()
    L.rl_q4_matvec(w, ws, x, y, T, N, K, group, x_scale=xs)
    assert torch.equal(y, first)
    for dt in (torch.float16, torch.bfloat16):
        z = torch.full((T, N), 2.0, dtype=dt, device="cuda")
        L.rl_q4_matvec(w, ws, x, z, T, N, K, group, x_scale=xs)
        assert torch.equal(z, first.to(dt))
    L.rl_q4_matvec(w, ws, x, y, T, N, K, group, x_scale=xs, accumulate=1)
    assert torch.all((y.double() - 2 * first.double()).abs() <= 2 * first.double().abs() * U)


@pytest.mark.parametrize("N,K,T,group", [(3000, 256, 75, 64), (2431, 512, 64, 128), (2433, 512, 65, 128), (40, 128, 129, 32)])
@pytest.mark.parametrize("xt", ["f8", "f32", "bf16"])
def test_q4_matvec_many_rows(L, N, K, T, group, xt):
    """Column groups that share a launch, with and without a rest, on both sides of 152 tiles."""
    w, ws, x, xs = q4_case(N, K, T, group, xt, seed=N)
    guard = torch.full((T * N + 64,), 3.0, device="cuda")
    y = guard[:T * N].view(T, N)
    L.rl_q4_matvec(w, ws, x, y, T, N, K, group, x_scale=xs)
    check_q4(y, *q4_ref(w, ws, x, xs, group), K, group, xt)
    assert torch.all(guard[T * N:] == 3.0)


def test_q4_matvec_extremes(L):
    """Smallest and largest nibbles, activations from 1e-38 to 1e30, zero rows and a token with a NaN
    beside healthy ones."""
    N, K, T, group = 48, 512, 6, 64
    w, ws, x, _ = q4_case(N, K, T, group, "f32", seed=4)
    w[0], w[1], w[2] = 0, 0x88, 0xff
    x[0] *= 1e-38
    x[1] *= 1e30
    x[2] = 0
    x[3, 100] = math.nan
    x[4, :64] *= 1e-20
    ref, mag, rep = q4_ref(w, ws, x, None, group)
    y = torch.empty(T, N, device="cuda")
    L.rl_q4_matvec(w, ws, x, y, T, N, K, group)
    ok = [0, 1, 2, 4, 5]
    assert torch.all(y[2] == 0) and torch.all(y[ok, 1] == 0) and y[3].isnan().all()
    n = 2 * 17 * 4 + 12 + 3 * 8 + 8
    bound = mag[ok] * (n * U + 2.0 ** -22) + rep[ok] * 2.0 ** -38 + 1e-42
    assert torch.all((y[ok].double() - ref[ok]).abs() <= bound)


# ---- rl_logprobs --------------------------------------------------------------------------
def lp_run(L, x, targets, n, ws=None):
    T, V = x.shape
    o = dict(logprob=torch.full((T,), 7.0, device="cuda"), entropy=torch.full((T,), 7.0, device="cuda"),
             ids=torch.full((T, n), -7, dtype=torch.int32, device="cuda") if n else None,
             top=torch.full((T, n), 7.0, device="cuda") if n else None)
    if ws is None:
        ws = torch.zeros(L.rl_logprobs_workspace_bytes(T, V, n), dtype=torch.uint8, device="cuda")
    L.rl_logprobs(x, T, V, targets, o["logprob"], o["entropy"], n, o["ids"], o["top"], ws, ws.numel())
    torch.cuda.synchronize()
    return o


def check_lp(o, x, targets, n):
    T, V = x.shape
    v = x.double()
    lp = torch.log_softmax(v, 1)
    # sums of positive terms: at most V / 256 + 64 per thread and merge chain; e^d by ex2 (2 u) of an
    # argument rounded once (|d| log2 e u); |d| counted up to 40, beyond it e^d vanishes
    s = (V / 256 + 64 + 2 + 60) * U
    want = lp.gather(1, targets.long()[:, None])[:, 0]
    assert torch.all((o["logprob"].double() - want).abs() <= s + 4 * U * (want.abs() + 1) + 4 * U * v.abs().amax())
    ent = -(lp.exp() * lp.nan_to_num(neginf=0.0)).sum(1)
    assert torch.all((o["entropy"].double() - ent).abs() <= s * (2 + ent) + 4 * U * (ent + 1))
    if n:
        ids = torch.from_numpy(np.argsort(-x.double().cpu().numpy(), axis=1, kind="stable")[:, :n].copy()).cuda()
        assert torch.equal(o["ids"].long(), ids)
        top = lp.gather(1, ids)
        assert torch.all((o["top"].double() - top).abs().nan_to_num(0.0) <= s + 4 * U * (top.abs().nan_to_num(posinf=0.0) + 1) + 4 * U * v.nan_to_num(neginf=0.0).abs().amax())


@pytest.mark.parametrize("T,V,n", [(1, 1, 1), (1, 131072, 20), (2, 4097, 32), (3, 33, 5), (1, 100003, 1), (5, 50001, 7),
                                   (40, 12289, 20), (700, 1000, 3), (16, 100003, 0), (4100, 77, 2),
                                   (9, 300001, 32), (500, 20011, 20), (3, 1000003, 17)])
@pytest.mark.parametrize("dt", list(TYPES))
def test_logprobs(L, T, V, n, dt):
    x = (3 * randn(T, V, seed=V)).to(TYPES[dt])
    targets = torch.randint(0, V, (T,), generator=torch.Generator().manual_seed(T)).to(torch.int32).cuda()
    check_lp(lp_run(L, x, targets, n), x, targets, n)


@pytest.mark.parametrize("V,T", [(4095, 456), (4096, 457), (4097, 228), (4097, 229), (16384, 114), (16384, 115),
                                 (62 * 4096 + 1, 7), (62 * 4096 + 1, 8), (63 * 4096, 7), (17, 456), (1, 1000)])
def test_logprobs_on_both_sides_of_a_split(L, V, T):
    """Rows in pieces of a tile (up to 456 pieces of at most 1/62 of a row) and in equal runs over all CTAs, V on
    both sides of a tile: every value belongs to exactly one piece.  A row's largest value marks a piece that
    is left out, the sums one that is counted twice."""
    n = min(V, 3)
    x = randn(T, V, seed=T)
    at = torch.randint(0, V, (T,), generator=torch.Generator().manual_seed(V)).cuda()
    x[torch.arange(T, device="cuda"), at] = 9.0
    x[: T // 2] = 0.5                                  # every value counts the same: log V
    check_lp(lp_run(L, x, at.to(torch.int32), n), x, at.to(torch.int32), n)


def test_logprobs_orders_that_defeat_a_threshold(L):
    """Rising, falling and equal rows, a row whose largest values share one thread's positions, ties
    across segments, signed zeros."""
    V, n = 40000, 32
    up = torch.arange(V, dtype=torch.float32) / 4000
    x = torch.stack([up, up.flip(0), torch.zeros(V), torch.zeros(V), torch.zeros(V), torch.randn(V)])
    x[3, ::1024] = 5
    x[4, 1::2] = -0.0
    x[5, 7::4096] = 6
    x = x.cuda()
    t = torch.tensor([0, 1, 39999, 5, 6, 7], dtype=torch.int32, device="cuda")
    check_lp(lp_run(L, x, t, n), x, t, n)
    big = x.repeat(300, 1)             # one segment per row
    check_lp(lp_run(L, big, t.repeat(300), n), big, t.repeat(300), n)


def test_logprobs_masked_and_non_finite_rows(L):
    V, n = 9001, 4
    x = randn(8, V, seed=6)
    x[0] = -math.inf                   # nothing left
    x[1] = -math.inf
    x[1, 8999] = 2.0                   # one token left
    x[2, 10:] = -math.inf
    x[3, 4500] = math.nan
    x[4, 17] = math.inf
    x[5] = torch.finfo(torch.float32).min
    x[6] = math.nan
    t = torch.tensor([3, 8999, 11, 5, 17, 100, 2, -1], dtype=torch.int32, device="cuda")
    o = lp_run(L, x, t, n)
    assert o["logprob"][:3].tolist() == [-math.inf, 0.0, -math.inf]
    assert o["entropy"][:2].tolist() == [0.0, 0.0]
    assert o["ids"][0].tolist() == [0, 1, 2, 3] and torch.all(o["top"][0] == -math.inf)
    assert o["ids"][1].tolist() == [8999, 0, 1, 2] and o["top"][1].tolist() == [0.0] + 3 * [-math.inf]
    for r in (3, 4, 6):
        assert o["logprob"][r].isnan() and o["entropy"][r].isnan() and o["top"][r].isnan().all()
    assert o["ids"][4][0] == 17 and o["ids"][6].tolist() == [0, 1, 2, 3]
    keep = x[3].clone()
    keep[4500] = -math.inf
    assert o["ids"][3].tolist() == keep.topk(4).indices.tolist()
    assert abs(float(o["logprob"][5]) + math.log(V)) < 1e-4 and abs(float(o["entropy"][5]) - math.log(V)) < 1e-4
    assert o["logprob"][7].isnan() and o["entropy"][7].isfinite()
    lp = torch.log_softmax(x[2].double(), 0)
    assert o["ids"][2].tolist() == x[2].topk(4).indices.tolist()
    assert abs(float(o["entropy"][2]) - float(-(lp.exp() * lp.clamp_min(-1e30)).sum())) < 1e-5


def test_logprobs_unaligned_rows_and_shared_workspace(L):
    """Rows that start off a 16-byte boundary; calls of different sizes in one workspace."""
    ws = torch.zeros(L.rl_logprobs_workspace_bytes(64, 70001, 32), dtype=torch.uint8, device="cuda")
    for T, V, n, dt in ((64, 70001, 32, "bf16"), (1, 70001, 4, "f32"), (5, 4099, 20, "f16"), (64, 70001, 32, "f32")):
        flat = randn(T * V + 3, seed=V + T, dtype=TYPES[dt])
        x = flat[1:1 + T * V].view(T, V)
        t = torch.randint(0, V, (T,), generator=torch.Generator().manual_seed(T)).to(torch.int32).cuda()
        check_lp(lp_run(L, x, t, n, ws), x, t, n)


def test_logprobs_each_output_alone(L):
    """Any of the outputs may be left out; the others keep their bits."""
    for T, V in ((3, 9001), (300, 20011)):
        x = 3 * randn(T, V, seed=V)
        t = torch.randint(0, V, (T,), generator=torch.Generator().manual_seed(T)).to(torch.int32).cuda()
        full = lp_run(L, x, t, 5)
        ws = torch.zeros(L.rl_logprobs_workspace_bytes(T, V, 5), dtype=torch.uint8, device="cuda")
        lp, en = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
        ids, top = torch.empty(T, 5, dtype=torch.int32, device="cuda"), torch.empty(T, 5, device="cuda")
        L.rl_logprobs(x, T, V, t, lp, None, 0, None, None, ws, ws.numel())
        L.rl_logprobs(x, T, V, None, None, en, 0, None, None, ws, ws.numel())
        L.rl_logprobs(x, T, V, None, None, None, 5, ids, top, ws, ws.numel())
        assert torch.equal(lp, full["logprob"]) and torch.equal(en, full["entropy"])
        assert torch.equal(ids, full["ids"]) and torch.equal(top, full["top"])


def test_logprobs_masked_vocabulary(L):
    """Most of every row masked, by -inf and by the type's lowest value, in 16 bits too."""
    T, V, n = 70, 30011, 8
    for dt in TYPES.values():
        x = (2 * randn(T, V, seed=8)).to(dt)
        x[:, 100:] = -math.inf
        x[1::2, 100:] = torch.finfo(dt).min
        t = torch.randint(0, 100, (T,), generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()
        o = lp_run(L, x, t, n)
        small = lp_run(L, x[:, :100].contiguous(), t, n)
        assert torch.equal(o["ids"], small["ids"])
        # the masked values add nothing, so that only the order of the sums differs
        for k in ("logprob", "entropy", "top"):
            assert torch.all((o[k] - small[k]).abs() <= 300 * U * (1 + small[k].abs())), k


@pytest.mark.parametrize("T,V,n", [(1, 250001, 1), (7, 250001, 1), (40, 12289, 16), (3, 9001, 20), (500, 20011, 5)])
def test_logprobs_merges_what_the_other_pieces_published(L, T, V, n):
    """Rows in pieces that one warp merges (at most 64 keys), call after call in one workspace without a wait
    between them: a merge that reads a piece before its CTA's publication is ordered sees the other input's
    triple or keys of the call before."""
    xs = [3 * randn(T, V, seed=V + i) - 5 * i for i in range(2)]
    t = torch.randint(0, V, (T,), generator=torch.Generator().manual_seed(T)).to(torch.int32).cuda()
    ws = torch.zeros(L.rl_logprobs_workspace_bytes(T, V, n), dtype=torch.uint8, device="cuda")
    want = [lp_run(L, x, t, n) for x in xs]
    for i in range(2):
        check_lp(want[i], xs[i], t, n)
    outs = [dict(logprob=torch.empty(T, device="cuda"), entropy=torch.empty(T, device="cuda"),
                 ids=torch.empty(T, n, dtype=torch.int32, device="cuda"), top=torch.empty(T, n, device="cuda"))
            for _ in range(100)]
    for i, o in enumerate(outs):
        L.rl_logprobs(xs[i % 2], T, V, t, o["logprob"], o["entropy"], n, o["ids"], o["top"], ws, ws.numel())
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        for k in o:
            assert torch.equal(o[k], want[i % 2][k]), (i, k)


@pytest.mark.parametrize("V", [131072, 1 << 20])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_logprobs_small_terms_beside_large_ones(L, V, dt):
    """4096 zeros (16 per thread of the row's CTA), then V - 4096 values whose terms lie below half a step of the
    sum of eight ones: added one by one to it they would all be lost, 1.4e-5 and 1.1e-4 of the sum.
    Bounds: of a sum of positive terms, the terms of a tile among themselves (7), the tiles, 2 values per
    lane, 5 + 5 shuffles and the merge of 2 pieces (7) make V / 4096 + 27 additions; the small terms'
    own error (|d| log2 e in the argument, 1.2 u each, and 4 u of ex2) counts with their share of S, below
    2^-13, and in full in U.  log S, U / S and the differences: 4 u of their magnitude, as in check_lp."""
    T, d = 456, -14.625
    x = torch.full((T, V), d, dtype=TYPES[dt], device="cuda")
    x[:, :4096] = 0
    t = torch.zeros(T, dtype=torch.int32, device="cuda")
    t[1::2] = V - 1
    o = lp_run(L, x, t, 0)
    e = math.exp(d)
    S, Um = 4096 + (V - 4096) * e, (V - 4096) * -d * e     # Um = -sum (x - m) e^(x - m)
    n = V / 4096 + 27
    rel_S = n * U + 2.0 ** -13 * (1.2 * -d + 4) * U
    want = torch.full((T,), -math.log(S), dtype=torch.float64, device="cuda")
    want[1::2] += d
    assert torch.all((o["logprob"].double() - want).abs() <= rel_S + 4 * U * (want.abs() + 1) + 4 * U * -d)
    entropy = math.log(S) + Um / S
    bound = rel_S + Um / S * (2 * n + 1.2 * -d + 4) * U + 4 * U * (entropy + 1)
    assert torch.all((o["entropy"].double() - entropy).abs() <= bound)


# ---- moe_decode_tokens --------------------------------------------------------------------
TINY = synth.WORKLOADS["tiny"]
SHAPES = {
    "tiny": TINY,
    "decode_layer": synth.WORKLOADS["decode_layer"],
    "one_expert": replace(TINY, top_k=1),
    "all_experts": replace(TINY, n_experts=16, top_k=16),
    "narrow": replace(TINY, hidden=256, n_experts=24, top_k=3, inter=256),
    "wide_inter": replace(TINY, hidden=1024, n_experts=20, top_k=8, inter=2048),
    "most_pairs": replace(TINY, hidden=512, n_experts=40, top_k=16, inter=1024),
    "odd_experts": replace(TINY, n_experts=157, top_k=5, inter=256),
    "widest": replace(TINY, hidden=2048, n_experts=12, top_k=8, inter=2048),
    "biased": replace(TINY, n_experts=64, zipf_s=1.1),
}


class Layer:
    """A one-layer model with the buffers of a step of T tokens."""

    def __init__(self, w):
        from quantized_moe_expert_rl_gb300 import engine
        self.engine, self.w = engine, w
        self.m = engine.Model(w, slot_perm=True)
        self.o = OracleSide(self.m)

    def run(self, L, x, stacked, y=None, accumulate=0, eps=None, ws=None):
        T = x.shape[0]
        b = self.engine.TokensBuffers.make(self.m, T)
        y = torch.full_like(x, 7.0) if y is None else y
        lg = torch.empty(T, self.w.n_experts, device="cuda")
        ws = b.ws if ws is None else ws
        L.moe_decode_tokens(self.m.shape, 0, T, x, 1e-6 if stacked else -1.0, self.m.routers[0],
                            None if self.m.bias is None else self.m.bias[0], self.m.table, self.m.codebook, b.ids[0],
                            b.weights[0], b.slots[0], b.miss, b.ctrl, lg, y, accumulate, ws, ws.numel())
        torch.cuda.synchronize()
        return b, lg, y

    def check(self, L, x, stacked=False):
        b, lg, y = self.run(L, x, stacked)
        assert b.ctrl.tolist() == [NO_EARLY_OUT, 0] and b.miss.tolist() == [0]
        xo = x.double().cpu().numpy()
        xn = oracle.rmsnorm(xo) if stacked else xo
        rep = {}
        r = check_route(lg.cpu().numpy(), b.ids[0].cpu().numpy(), b.weights[0].cpu().numpy(), u64(b.slots[0]),
                        oracle.router_logits(xn, self.o.router(0), self.o.bias(0)), self.o.table_row(0), self.w.top_k, 0, rep)
        assert rep["near_ties"] == 0
        assert rel_l2(y.cpu().numpy(), self.o.experts(xn, r.ids, r.weights, r.slots)) <= REL_F32
        return b, y


@pytest.fixture(scope="module", params=list(SHAPES))
def layer(request, L):
    return Layer(SHAPES[request.param])


def rows(w, T, seed=1):
    return randn(T, w.hidden, seed=seed)


@pytest.mark.parametrize("T", [1, 2, 3, 7, 32])
def test_moe_tokens(L, layer, T):
    x = rows(layer.w, T, seed=T)
    layer.check(L, x, stacked=False)
    b, y = layer.check(L, x, stacked=True)
    # the same call again, and each token's result whatever its company
    b2, _, y2 = layer.run(L, x, True)
    assert torch.equal(y2, y) and torch.equal(b2.ids, b.ids)
    _, _, y1 = layer.run(L, x[T - 1:].contiguous(), True)
    assert torch.equal(y1[0], y[T - 1])


def test_moe_tokens_shared_experts(L, layer):
    """Equal tokens (every expert serves all of them) and near-equal ones."""
    x = rows(layer.w, 1, seed=9).repeat(32, 1)
    _, y = layer.check(L, x)
    assert torch.equal(y, y[:1].expand(32, -1))
    x = x[:11] + 0.05 * rows(layer.w, 11, seed=10)
    layer.check(L, x, stacked=True)


def test_moe_tokens_accumulates_into_its_input(L, layer):
    x = rows(layer.w, 5, seed=3)
    _, _, y = layer.run(L, x, True)
    z = x.clone()
    layer.run(L, z, True, y=z, accumulate=1)
    assert torch.equal(z, x + y)
    z = x.clone()
    layer.run(L, z, True, y=z)
    assert torch.equal(z, y)


@pytest.fixture(scope="module")
def small(L):
    return Layer(TINY)


def test_moe_tokens_magnitudes(L, small):
    """Rows of very different size side by side: each keeps its own accuracy."""
    x = rows(TINY, 6, seed=5)
    x[1] *= 1e-12
    x[2] *= 300
    x[3] = 0
    x[4, 1:] = 0
    b, lg, y = small.run(L, x, False)
    xo = x.double().cpu().numpy()
    ids, wt = b.ids[0].cpu().numpy(), b.weights[0].double().cpu().numpy()
    ref = small.o.experts(xo, ids, wt, u64(b.slots[0]))
    for t in range(6):
        if t == 3:
            assert torch.all(y[3] == 0)
        else:
            assert rel_l2(y[t].cpu().numpy(), ref[t]) <= REL_F32, t
    assert b.ids[0][3].tolist() == [0, 1, 2, 3]          # equal logits: lowest indices


def test_moe_tokens_one_workspace_for_all_sizes(L, small):
    ws = torch.zeros(L.moe_decode_tokens_workspace_bytes(small.m.shape, 32), dtype=torch.uint8, device="cuda")
    for T in (32, 1, 5, 32, 2):
        x = rows(TINY, T, seed=T + 50)
        _, _, y = small.run(L, x, True, ws=ws)
        assert torch.equal(y, small.run(L, x, True)[2])


def test_moe_tokens_misses_and_given_routing(L):
    w = replace(TINY, n_resident=20)
    s = Layer(w)
    x = rows(w, 6, seed=8)
    b, lg, y = s.run(L, x, True)
    ids = b.ids[0].cpu().numpy()
    absent = sorted({int(e) for e in ids.flatten() if not s.m.resident[0, e]})
    misses = sum(not s.m.resident[0, e] for e in ids.flatten())
    assert misses > 0 and b.ctrl.tolist() == [0, 0] and b.miss.tolist() == [misses]
    assert torch.all(y == 7.0)                             # untouched
    assert [int(v) == 0 for v in b.slots[0].flatten()] == [not s.m.resident[0, e] for e in ids.flatten()]
    call = lambda: L.moe_decode_tokens(s.m.shape, 0, 6, x, 1e-6, None, None, None, s.m.codebook, b.ids[0],  # noqa: E731
                                       b.weights[0], b.slots[0], None, b.ctrl, None, y, 0, b.ws, b.ws.numel())
    call()                                                # the flag stops it
    torch.cuda.synchronize()
    assert torch.all(y == 7.0) and b.ctrl.tolist() == [0, 0]
    b.ctrl[0] = NO_EARLY_OUT
    call()                                                # absent slots are refused on the device
    torch.cuda.synchronize()
    assert torch.all(y == 7.0) and b.ctrl.tolist() == [NO_EARLY_OUT, L.RL_DEVERR_MISSING]
    b.ctrl[1] = 0
    s.m.fill(0, absent)
    L.rl_resolve_slots(s.m.shape, 0, 6, b.ids[0], s.m.table, b.slots[0])
    call()
    torch.cuda.synchronize()
    assert b.ctrl.tolist() == [NO_EARLY_OUT, 0]
    full = s.run(L, x, True)
    assert torch.equal(full[0].ids, b.ids) and torch.equal(full[2], y)
    for at, bit, bad in ((b.ids, L.RL_DEVERR_BAD_ID, w.n_experts), (b.ids, L.RL_DEVERR_BAD_ID, -1),
                         (b.slots, L.RL_DEVERR_SLOT_ALIGN, int(b.slots[0, 2, 1]) + 4)):
        keep = at.clone()
        at[0, 2, 1] = bad
        y.fill_(7.0)
        call()
        torch.cuda.synchronize()
        assert torch.all(y == 7.0) and b.ctrl.tolist() == [NO_EARLY_OUT, bit]
        b.ctrl[1] = 0
        at.copy_(keep)


def test_moe_tokens_given_routing_may_repeat_an_expert(L, small):
    """The same expert twice in a token's list, as moe_decode takes it: both weights count."""
    x = rows(TINY, 3, seed=14)
    b, _, _ = small.run(L, x, False)
    b.ids[0, 1, 2] = b.ids[0, 1, 0]
    b.slots[0, 1, 2] = b.slots[0, 1, 0]
    y = torch.empty_like(x)
    small.engine.enqueue_tokens_layer(small.m, b, 0, x, y, stacked=False, routed=False)
    torch.cuda.synchronize()
    ref = small.o.experts(x.double().cpu().numpy(), b.ids[0].cpu().numpy(), b.weights[0].double().cpu().numpy(),
                          u64(b.slots[0]))
    assert b.ctrl.tolist() == [NO_EARLY_OUT, 0] and rel_l2(y.cpu().numpy(), ref) <= REL_F32


def test_moe_tokens_norm_range_is_flagged(L, small):
    """Beyond the fixed-point range of the RMSNorm's squares the call says so, as rl_route does."""
    x = rows(TINY, 3, seed=15)
    x[2] *= 1e4
    b, _, _ = small.run(L, x, True)
    assert b.ctrl.tolist() == [NO_EARLY_OUT, L.RL_DEVERR_RANGE]
    b, _, _ = small.run(L, x, False)
    assert b.ctrl.tolist() == [NO_EARLY_OUT, 0]


def test_moe_tokens_nan_router_is_flagged(L, small):
    x = rows(TINY, 3, seed=4)
    x[1, 5] = math.nan
    b, _, _ = small.run(L, x, False)
    assert b.ctrl[1] == L.RL_DEVERR_NAN


def test_moe_tokens_early_out_skips(L, small):
    x = rows(TINY, 3, seed=4)
    b = small.engine.TokensBuffers.make(small.m, 3)
    b.ctrl[0] = -1
    y = torch.full_like(x, 7.0)
    small.engine.enqueue_tokens_layer(small.m, b, 0, x, y, stacked=False)
    torch.cuda.synchronize()
    assert torch.all(y == 7.0) and torch.all(b.ids == 0) and b.ctrl.tolist() == [-1, 0]


def test_moe_tokens_waits_run_out(L, small):
    """A CTA held back (the test knob in the workspace header): the others' wait ends with an error
    status and nothing is written; the next call on a re-zeroed workspace is undisturbed."""
    x = rows(TINY, 4, seed=12)
    want = small.run(L, x, True)[2]
    ws = torch.zeros(L.moe_decode_tokens_workspace_bytes(small.m.shape, 4), dtype=torch.uint8, device="cuda")
    ws[64:72] = torch.tensor([20000, 3], dtype=torch.int32).view(torch.uint8).cuda()
    b, _, y = small.run(L, x, True, ws=ws)
    assert b.ctrl[1] == L.RL_DEVERR_WAIT_TIMEOUT and torch.all(y == 7.0)
    ws.zero_()
    b, _, y = small.run(L, x, True, ws=ws)
    assert b.ctrl.tolist() == [NO_EARLY_OUT, 0] and torch.equal(y, want)


def test_moe_tokens_agrees_with_single_token_decode(L):
    """Beside moe_decode_layer at the decode shape: the same experts, outputs within both bounds."""
    s = Layer(synth.WORKLOADS["decode_layer"])
    x = rows(s.w, 4, seed=21)
    b, _, y = s.run(L, x, False)
    d = s.engine.DecodeBuffers.make(s.m)
    for t in range(4):
        z = torch.zeros(s.w.hidden, device="cuda")
        s.engine.enqueue_decode_layer_fused(s.m, d, x[t], z)
        torch.cuda.synchronize()
        assert torch.equal(d.ids[0], b.ids[0, t])
        assert rel_l2(y[t].cpu().numpy(), z.cpu().numpy()) <= 2 * REL_F32


# ---- the operators together ---------------------------------------------------------------
def verify_ref(s, head, x, y_layers, targets, n):
    """From the GPU's residual stream after the layers: norm, head and log probabilities in 64 bits
    (the 8-bit row and its scales are taken as the GPU wrote them)."""
    T, H = x.shape
    v = head.q.double().view(T, H // head.group, head.group) * head.q_scale.double()[..., None]
    q = torch.stack((head.w & 15, head.w >> 4), 2).view(head.w.shape[0], H).double() - 8
    return v.view(T, H) @ (q * head.scale.double().repeat_interleave(head.group, 1)).t()


@pytest.mark.parametrize("T", [1, 5])
def test_verify_step(L, T):
    """Layers, norm, head and log probabilities as a verification step runs them, eagerly and as
    a captured graph replayed on new tokens."""
    from quantized_moe_expert_rl_gb300 import engine
    w = replace(TINY, n_layers=3)
    m = engine.Model(w)
    o = OracleSide(m)
    V, n = 5003, 6
    gain = 1 + 0.1 * randn(w.hidden, seed=31)
    head = engine.Head.make(0.05 * randn(V, w.hidden, seed=32), T, gain=gain, group=64, top_n=n)
    b = engine.TokensBuffers.make(m, T)
    x, y = torch.empty(T, w.hidden, device="cuda"), torch.empty(T, w.hidden, device="cuda")
    targets = torch.zeros(T, dtype=torch.int32, device="cuda")
    graph = None
    for step in range(3):
        x.copy_(rows(w, T, seed=40 + step))
        targets.copy_(torch.randint(0, V, (T,), generator=torch.Generator().manual_seed(step)).to(torch.int32))
        if step == 0:
            engine.enqueue_verify(m, b, head, x, y, targets)
        elif graph is None:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                engine.enqueue_verify(m, b, head, x, y, targets)
            graph.replay()
        else:
            graph.replay()
        torch.cuda.synchronize()
        assert b.ctrl.tolist() == [NO_EARLY_OUT, 0]
        # the layers, each from the oracle's own stream
        xo = x.double().cpu().numpy()
        for l in range(m.L):
            xn = oracle.rmsnorm(xo)
            r = oracle.route(xn, synth.router(w, l), None, m.table_host[l], w.top_k, l)
            assert np.array_equal(r.ids, b.ids[l].cpu().numpy())
            xo = xo + o.experts(xn, r.ids, r.weights, r.slots)
        assert rel_l2(y.cpu().numpy(), xo) <= m.L * REL_F32
        _, v = norm_ref(y, None, gain, 1e-6, torch.float32)
        back = head.q.double().view(T, -1, 64) * head.q_scale.double()[..., None]
        assert rel_l2(back.view(T, -1).cpu().numpy(), v.cpu().numpy()) <= 2.0 ** -4
        lg = verify_ref(m, head, x, y, targets, n)
        assert rel_l2(head.logits.cpu().numpy(), lg.cpu().numpy()) <= REL_F32
        check_lp(dict(logprob=head.logprob, entropy=head.entropy, ids=head.top_ids, top=head.top_logprob), head.logits,
                 targets, n)


def test_smaller_steps_in_the_same_buffers(L):
    """Steps of any number of tokens up to the buffers' in one set of buffers: the bits of a step in buffers of
    its own size, and the rows behind it left as they were."""
    from quantized_moe_expert_rl_gb300 import engine
    w = replace(TINY, n_layers=2)
    m = engine.Model(w)
    weight, n = 0.05 * randn(1009, w.hidden, seed=33), 4
    b, head = engine.TokensBuffers.make(m, 7), engine.Head.make(weight, 7, group=64, top_n=n)
    for T in (7, 1, 4, 0, 7, 3):
        x = rows(w, T, seed=80 + T) if T else torch.empty(0, w.hidden, device="cuda")
        t = torch.arange(T, dtype=torch.int32, device="cuda")
        outs = (head.logits, head.logprob, head.entropy, head.top_ids, head.top_logprob)
        for o in outs:
            o.fill_(7)
        ids = b.ids.clone()
        y = torch.empty_like(x)
        engine.enqueue_verify(m, b, head, x, y, t)
        torch.cuda.synchronize()
        assert b.ctrl.tolist() == [NO_EARLY_OUT, 0] and torch.equal(b.ids[:, T:], ids[:, T:])
        assert all(torch.all(o[T:] == 7) for o in outs)
        if T == 0:
            continue
        b1, h1 = engine.TokensBuffers.make(m, T), engine.Head.make(weight, T, group=64, top_n=n)
        z = torch.empty_like(x)
        engine.enqueue_verify(m, b1, h1, x, z, t)
        torch.cuda.synchronize()
        assert torch.equal(z, y) and torch.equal(b1.ids, b.ids[:, :T])
        for o, o1 in zip(outs, (h1.logits, h1.logprob, h1.entropy, h1.top_ids, h1.top_logprob)):
            assert torch.equal(o[:T], o1)


def test_bounded_tokens_match_full_residency(L):
    from quantized_moe_expert_rl_gb300 import engine
    w = replace(TINY, n_layers=4, n_resident=24)
    m, full = engine.Model(w), engine.Model(replace(w, n_resident=-1))
    T = 5
    b, bf = engine.TokensBuffers.make(m, T), engine.TokensBuffers.make(full, T)
    for step in range(2):
        x = rows(w, T, seed=60 + step)
        y, yf = torch.empty_like(x), torch.empty_like(x)
        b.miss.zero_()
        st = engine.run_bounded_tokens(m, b, x, y)
        engine.enqueue_tokens(full, bf, x, yf)
        torch.cuda.synchronize()
        assert torch.equal(y, yf) and torch.equal(b.ids, bf.ids)
        assert (step > 0 or st.early_outs) and b.ctrl[1] == 0
        for l in range(w.n_layers):
            assert (int(b.miss[l]) > 0) == (l in st.early_outs)


def test_other_stream(L, small):
    """Called on a stream of its own, after work on it."""
    x = rows(TINY, 4, seed=70)
    want = small.run(L, x, True)[2]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b = small.engine.TokensBuffers.make(small.m, 4)
    x2 = torch.zeros_like(x)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        x2.copy_(x)
        small.engine.enqueue_tokens_layer(small.m, b, 0, x2, x2, stacked=True)
    s.synchronize()
    assert torch.equal(x2, x + want) and b.ctrl.tolist() == [NO_EARLY_OUT, 0]
