"""rl_f8_matmul and rl_f8_gated on the GPU against plain computations in 64 bits.

Bounds.  u = 2^-24 is half a step of f32.  The products of two e4m3 values are exact in f32.  A block of 128
of them is added in f32 (two steps of rounding or truncation, 2 u, allowed for each of 128 additions), a
block's sum is multiplied by the rounded product of two scales and added to the sum of the blocks before it,
at most KB + 8 additions.  So a sum is off by at most (256 + KB + 8 + 4) u of the sum of magnitudes; half a step of
the result's type is added where it is rounded (eps / 2 relative; half of the smallest subnormal)."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from tests._gpu_common import REL_F32, rel_l2  # noqa: E402

U = 2.0 ** -24
F8 = torch.float8_e4m3fn
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def L():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from quantized_moe_expert_rl_gb300 import _lib, build
    build.build()
    return _lib


def blocks(n):
    return -(-n // 128)


def rows(T, K, g, spread=3.0):
    """Rows in 8 bits over most of the type's range, with scales of their own for every 128."""
    x = (torch.randn(T, K, generator=g) * 2.0 ** (spread * torch.randn(T, K, generator=g))).clamp(-448, 448).to(F8)
    return x.cuda(), (0.5 + torch.rand(T, blocks(K), generator=g)).cuda()


def matrix(N, K, g):
    w = (60 * torch.randn(N, K, generator=g)).clamp(-448, 448).to(F8)
    return w.cuda(), ((0.5 + torch.rand(blocks(N), blocks(K), generator=g)) * 1e-3).cuda()


def full(v, s, rows_per=1):
    """Values in 64 bits with their scales."""
    N, K = v.shape
    return v.double() * s.double().repeat_interleave(rows_per, 0)[:N].repeat_interleave(128, 1)[:, :K]


def reference(x, xs, w, ws):
    """(product, bound of its error)"""
    a, b = full(x, xs), full(w, ws, 128)
    return a @ b.t(), (a.abs() @ b.abs().t()) * (256 + blocks(x.shape[1]) + 12) * U


def rounding(dt):
    f = torch.finfo(dt)
    return (0.0 if dt == torch.float32 else f.eps / 2), (0.0 if dt == torch.float32 else f.smallest_normal * f.eps)


def close(y, ref, err, dt):
    rel, tiny = rounding(dt)
    assert y.dtype == dt
    bad = (y.double() - ref).abs() > err * (1 + rel) + ref.abs() * (rel + U) + tiny
    assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()} out of bounds"


SIZES = [(1, 1, 16), (1, 512, 2048), (1, 2048, 512), (2, 130, 144), (3, 127, 128), (8, 1000, 1040), (16, 257, 400),
         (17, 640, 2048), (31, 96, 48), (33, 129, 272), (50, 1016, 784), (64, 128, 8192), (65, 384, 128), (77, 1007, 1040),
         (128, 300, 640), (129, 300, 640), (200, 255, 112), (256, 513, 1040), (300, 2048, 512), (1000, 130, 4096),
         (130, 20000, 128), (5, 40000, 256), (70, 45000, 128)]


@pytest.mark.parametrize("T,N,K", SIZES)
def test_f8_matmul(L, T, N, K):
    g = torch.Generator().manual_seed(T * 1000003 + N * 1009 + K)
    x, xs = rows(T, K, g)
    w, ws = matrix(N, K, g)
    ref, err = reference(x, xs, w, ws)
    for name, dt in TYPES.items():
        y = torch.full((T, N), 7.0, dtype=dt, device="cuda")
        L.rl_f8_matmul(w, ws, x, xs, y, T, N, K)
        close(y, ref, err, dt)
        res = torch.randn(T, N, generator=g).to(dt).cuda()
        y2, keep = torch.full_like(y, 7), res.clone()
        L.rl_f8_matmul(w, ws, x, xs, y2, T, N, K, res=res)
        close(y2, ref + res.double(), err + (ref + res.double()).abs() * U, dt)
        assert torch.equal(res, keep)
        L.rl_f8_matmul(w, ws, x, xs, res, T, N, K, res=res)  # in place
        assert torch.equal(res, y2)
        if name == "f32":
            assert rel_l2(y.double().cpu().numpy(), ref.cpu().numpy()) <= REL_F32


GATED = [(1, 512, 2048), (1, 16, 16), (2, 130, 144), (5, 127, 128), (16, 1016, 784), (17, 256, 2048), (33, 129, 272),
         (50, 1016, 784), (64, 512, 2048), (65, 512, 2048), (129, 300, 640), (257, 640, 1040), (300, 1000, 128), (9, 25000, 64),
         (40, 22000, 64)]


@pytest.mark.parametrize("T,I,K", GATED)
def test_f8_gated(L, T, I, K):
    g = torch.Generator().manual_seed(T * 1000003 + I * 1009 + K)
    x, xs = rows(T, K, g, spread=1.0)
    (wg, sg), (wu, su) = matrix(I, K, g), matrix(I, K, g)
    sg *= 4 / (xs.mean() * 60 * 1e-3 * K ** 0.5 * 3)  # gates of a few units
    a, da = reference(x, xs, wg, sg)
    b, db = reference(x, xs, wu, su)
    ref = a * torch.sigmoid(a) * b
    # |silu'| < 1.1; exp, the sum, the division and the product: 8 half steps
    err = 1.1 * da * b.abs() + (a * torch.sigmoid(a)).abs() * db + 1.1 * da * db + 8 * U * ref.abs()
    for dt in TYPES.values():
        h = torch.full((T, I), 7.0, dtype=dt, device="cuda")
        L.rl_f8_gated(wg, sg, wu, su, x, xs, T, I, K, h=h)
        close(h, ref, err, dt)
    q, scale = torch.zeros(T, I, dtype=F8, device="cuda"), torch.full((T, blocks(I)), 7.0, device="cuda")
    h2 = torch.full((T, I), 7.0, device="cuda")
    L.rl_f8_gated(wg, sg, wu, su, x, xs, T, I, K, h=h2, q=q, scale=scale)
    q1, s1 = torch.zeros_like(q), torch.zeros_like(scale)
    L.rl_f8_gated(wg, sg, wu, su, x, xs, T, I, K, q=q1, scale=s1)
    assert torch.equal(q1.view(torch.uint8), q.view(torch.uint8)) and torch.equal(s1, scale)
    # (q, scale) against the f32 values that they stand for: the scale is two roundings off, a quotient three
    # (of the factor and of the product), then half a step of e4m3, below its smallest normal 2^-10 of the scale
    pad = torch.nn.functional.pad(h2.double(), (0, -I % 128)).view(T, -1, 128)
    top = pad.abs().amax(2)
    assert torch.all((scale.double() - top / 448).abs() <= 2 * U * top / 448)
    back = full(q, scale)
    assert torch.all((back - h2.double()).abs() <= h2.double().abs() * (2.0 ** -4 + 8 * U)
                     + 2.0 ** -10 * 1.001 * scale.double().repeat_interleave(128, 1)[:, :I])


@pytest.mark.parametrize("T", [1, 20, 100, 300])
def test_f8_broken_values_stay_in_their_row(L, T):
    """NaN and infinite scales and an e4m3 NaN reach their own token's outputs only; the other rows keep their bits."""
    N, K = 640, 400
    g = torch.Generator().manual_seed(T)
    x, xs = rows(T, K, g)
    (w, ws), (wu, su) = matrix(N, K, g), matrix(N, K, g)
    good, q, s = torch.empty(T, N, device="cuda"), torch.zeros(T, N, dtype=F8, device="cuda"), torch.zeros(T, 5, device="cuda")
    L.rl_f8_matmul(w, ws, x, xs, good, T, N, K)
    L.rl_f8_gated(w, ws, wu, su, x, xs, T, N, K, q=q, scale=s)
    bad = torch.tensor(sorted({0, T // 2, T - 1}))
    x2, xs2 = x.clone(), xs.clone()
    xs2[bad[0], 1] = float("nan")
    x2.view(torch.uint8)[bad[-1], 7] = 0x7F
    if len(bad) > 2:
        xs2[bad[1], 3] = float("inf")
    y, q2, s2 = torch.empty_like(good), torch.ones_like(q), torch.ones_like(s)
    L.rl_f8_matmul(w, ws, x2, xs2, y, T, N, K)
    L.rl_f8_gated(w, ws, wu, su, x2, xs2, T, N, K, q=q2, scale=s2)
    rest = torch.ones(T, dtype=torch.bool)
    rest[bad] = False
    assert torch.equal(y[rest], good[rest]) and torch.equal(s2[rest], s[rest])
    assert torch.equal(q2.view(torch.uint8)[rest], q.view(torch.uint8)[rest])
    assert not torch.isfinite(y[bad]).any()
    assert torch.isnan(s2[bad]).all() and (q2.float()[bad] == 0).all()  # a group with a NaN or an infinity is marked


@pytest.mark.parametrize("T", [3, 200])
def test_f8_zeros_and_extremes(L, T):
    """Zero rows, zero scales and zero weights give zeros (scale 0, q 0); the type's largest values everywhere."""
    N, K = 300, 256
    z8 = lambda *s: torch.zeros(*s, device="cuda").to(F8)  # noqa: E731
    one, big = torch.ones(T, 2, device="cuda"), torch.full((T, K), 448.0, device="cuda").to(F8)
    w1, wbig = torch.ones(3, 2, device="cuda"), torch.full((N, K), 448.0, device="cuda").to(F8)
    y = torch.full((T, N), 7.0, device="cuda")
    q, s = torch.ones(T, N, dtype=F8, device="cuda"), torch.full((T, 3), 7.0, device="cuda")
    for x, xs, w, ws in ((z8(T, K), one, wbig, w1), (big, 0 * one, wbig, w1), (big, one, z8(N, K), w1), (big, one, wbig, 0 * w1)):
        L.rl_f8_matmul(w, ws, x, xs, y, T, N, K)
        L.rl_f8_gated(w, ws, w, ws, x, xs, T, N, K, q=q, scale=s)
        assert not y.any() and not s.any() and not q.float().any()
    L.rl_f8_matmul(wbig, w1, big, one, y, T, N, K)
    assert torch.equal(y, torch.full_like(y, 448.0 * 448.0 * K))  # exact in f32
    # silu(v) v with v = 448^2 K up to f32's largest: finite, at the top of the type
    L.rl_f8_gated(wbig, w1, wbig, w1, big, one, T, N, K, q=q, scale=s)
    assert (q.float() == 448).all() and torch.isfinite(s).all()
    # values near the smallest subnormal: 448 / max leaves f32's range
    L.rl_f8_gated(wbig, w1, wbig, w1 * 1e-33, big, one * 1e-6, T, N, K, q=q, scale=s)
    assert torch.isfinite(q.float()).all() and torch.isfinite(s).all() and (s > 0).all()
    assert (q.float() > 400).all()


def test_f8_rows_apart_from_16_bytes(L):
    """Outputs and residuals at any element, sizes that no vector divides."""
    g = torch.Generator().manual_seed(3)
    for T, N, K in ((5, 129, 144), (200, 515, 144), (150, 513, 272)):
        x, xs = rows(T, K, g)
        w, ws = matrix(N, K, g)
        ref, err = reference(x, xs, w, ws)
        for dt in TYPES.values():
            y = torch.zeros(T * N + 3, dtype=dt, device="cuda")[3:].view(T, N)
            res = torch.randn(T * N + 1, generator=g).to(dt).cuda()[1:].view(T, N)
            L.rl_f8_matmul(w, ws, x, xs, y, T, N, K, res=res)
            close(y, ref + res.double(), err + (ref + res.double()).abs() * U, dt)


@pytest.mark.parametrize("T", [2, 60, 140])
def test_f8_skips_a_stopped_layer(L, T):
    """ctrl[0] <= layer: nothing is written; above it the call runs.  No error bits either way."""
    g = torch.Generator().manual_seed(T)
    x, xs = rows(T, 256, g)
    w, ws = matrix(300, 256, g)
    ctrl = torch.tensor([5, 0], dtype=torch.int32, device="cuda")
    y = torch.full((T, 300), 7.0, device="cuda")
    q, s = torch.ones(T, 300, dtype=F8, device="cuda"), torch.full((T, 3), 7.0, device="cuda")
    for layer in (5, 6):
        L.rl_f8_matmul(w, ws, x, xs, y, T, 300, 256, layer=layer, ctrl=ctrl)
        L.rl_f8_gated(w, ws, w, ws, x, xs, T, 300, 256, q=q, scale=s, layer=layer, ctrl=ctrl)
    assert (y == 7).all() and (s == 7).all() and (q.float() == 1).all()
    L.rl_f8_matmul(w, ws, x, xs, y, T, 300, 256, layer=4, ctrl=ctrl)
    L.rl_f8_gated(w, ws, w, ws, x, xs, T, 300, 256, q=q, scale=s, layer=4, ctrl=ctrl)
    ref, err = reference(x, xs, w, ws)
    close(y, ref, err, torch.float32)
    assert (s != 7).all() and ctrl.tolist() == [5, 0]


@pytest.mark.parametrize("T", [1, 30, 300])
def test_f8_graph_stream_and_neighbours(L, T):
    """Captured and replayed on new rows; another stream; two calls side by side; the bytes behind the outputs."""
    N, K = 1030, 512
    g = torch.Generator().manual_seed(T)
    w, ws = matrix(N, K, g)
    x, xs = rows(T, K, g)
    buf = torch.full((T * N + 64,), 7.0, device="cuda")
    y = buf[:T * N].view(T, N)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    ys = [torch.empty(T, N, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    for s, out in zip((s1, s2), ys):
        for _ in range(5):
            L.rl_f8_matmul(w, ws, x, xs, out, T, N, K, stream=s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.rl_f8_matmul(w, ws, x, xs, y, T, N, K)
    for k in range(3):
        x2, xs2 = rows(T, K, g)
        x.copy_(x2), xs.copy_(xs2)
        graph.replay()
        torch.cuda.synchronize()
        ref, err = reference(x, xs, w, ws)
        close(y, ref, err, torch.float32)
    assert (buf[T * N:] == 7).all() and torch.equal(ys[0], ys[1])


@pytest.mark.parametrize("T,N,K,calls", [(8, 60000, 2048, 400), (1, 2048, 512, 2000), (40, 20000, 1040, 300), (77, 10007, 1040, 300),
                                         (200, 4096, 1024, 300)])
def test_f8_repeats(L, T, N, K, calls):
    """Many calls back to back, several tiles per CTA: the same bits every time, no error bits."""
    g = torch.Generator().manual_seed(N)
    x, xs = rows(T, K, g)
    w, ws = matrix(N, K, g)
    ctrl = torch.tensor([0x7FFFFFFF, 0], dtype=torch.int32, device="cuda")
    first, y, odd = torch.empty(T, N, device="cuda"), torch.empty(T, N, device="cuda"), torch.zeros(1, dtype=torch.int64, device="cuda")
    L.rl_f8_matmul(w, ws, x, xs, first, T, N, K, ctrl=ctrl)
    for _ in range(calls):
        y.fill_(7)
        L.rl_f8_matmul(w, ws, x, xs, y, T, N, K, ctrl=ctrl)
        odd += (y != first).sum()
    ref, err = reference(x, xs, w, ws)
    close(first, ref, err, torch.float32)
    assert int(odd) == 0 and ctrl.tolist() == [0x7FFFFFFF, 0]


@pytest.mark.parametrize("T,N,K", [(1100, 20000, 272), (1100, 20000, 640), (600, 30001, 1040), (70, 45000, 400)])
def test_f8_matmul_tiles_after_tiles(L, T, N, K):
    """Three tiles and more for every CTA or pair, odd numbers of blocks: what is kept between blocks goes on across tiles."""
    g = torch.Generator().manual_seed(N + K)
    x, xs = rows(T, K, g)
    w, ws = matrix(N, K, g)
    ref, err = reference(x, xs, w, ws)
    y = torch.full((T, N), 7.0, dtype=torch.bfloat16, device="cuda")
    L.rl_f8_matmul(w, ws, x, xs, y, T, N, K)
    close(y, ref, err, torch.bfloat16)


@pytest.mark.parametrize("T,I,K,calls", [(600, 13000, 272, 60), (600, 13000, 640, 60), (300, 20001, 1040, 60), (2048, 512, 2048, 500),
                                         (40, 22000, 400, 100), (1, 512, 2048, 1000)])
def test_f8_gated_tiles_after_tiles(L, T, I, K, calls):
    """The gated form over several tiles per CTA or pair, and called many times: right, and the same bits every time."""
    g = torch.Generator().manual_seed(I + K)
    x, xs = rows(T, K, g, spread=1.0)
    (wg, sg), (wu, su) = matrix(I, K, g), matrix(I, K, g)
    sg *= 4 / (xs.mean() * 60 * 1e-3 * K ** 0.5 * 3)  # gates of a few units
    a, da = reference(x, xs, wg, sg)
    b, db = reference(x, xs, wu, su)
    ref = a * torch.sigmoid(a) * b
    err = 1.1 * da * b.abs() + (a * torch.sigmoid(a)).abs() * db + 1.1 * da * db + 8 * U * ref.abs()  # as in test_f8_gated
    h = torch.full((T, I), 7.0, device="cuda")
    q, scale = torch.zeros(T, I, dtype=F8, device="cuda"), torch.full((T, blocks(I)), 7.0, device="cuda")
    ctrl = torch.tensor([0x7FFFFFFF, 0], dtype=torch.int32, device="cuda")
    L.rl_f8_gated(wg, sg, wu, su, x, xs, T, I, K, h=h, q=q, scale=scale, ctrl=ctrl)
    close(h, ref, err, torch.float32)
    top = torch.nn.functional.pad(h.double(), (0, -I % 128)).view(T, -1, 128).abs().amax(2)
    assert torch.all((scale.double() - top / 448).abs() <= 2 * U * top / 448)
    assert torch.all((full(q, scale) - h.double()).abs() <= h.double().abs() * (2.0 ** -4 + 8 * U)
                     + 2.0 ** -10 * 1.001 * scale.double().repeat_interleave(128, 1)[:, :I])
    odd = torch.zeros(1, dtype=torch.int64, device="cuda")
    q1, s1 = torch.empty_like(q), torch.empty_like(scale)
    for _ in range(calls):
        q1.view(torch.uint8).fill_(1), s1.fill_(7)
        L.rl_f8_gated(wg, sg, wu, su, x, xs, T, I, K, q=q1, scale=s1, ctrl=ctrl)
        odd += (q1.view(torch.uint8) != q.view(torch.uint8)).sum() + (s1 != scale).sum()
    assert int(odd) == 0 and ctrl.tolist() == [0x7FFFFFFF, 0]
