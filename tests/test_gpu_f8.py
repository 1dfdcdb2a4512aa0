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
