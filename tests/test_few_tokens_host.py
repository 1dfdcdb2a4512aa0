"""The operators of a step of a few tokens (moe_decode_tokens, rl_add_rmsnorm, rl_q4_matvec,
rl_logprobs): refusals made on the host before any launch, and the packing of 4-bit weights.  No
GPU needed."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    from quantized_moe_expert_rl_gb300 import _lib, build
    build.build()
    return _lib.load()


INVALID, UNSUPPORTED = 1, 2
FAKE, ODD = ctypes.c_void_p(1 << 20), ctypes.c_void_p((1 << 20) + 2)


def _with(args, **changes):
    out = dict(args)
    out.update(changes)
    return list(out.values())


def test_moe_decode_tokens_refusals(lib):
    from quantized_moe_expert_rl_gb300._lib import RlShape
    s = RlShape.of(2048, 512, 10, 512, 4)
    need = lib.moe_decode_tokens_workspace_bytes(ctypes.byref(s), 32)
    assert need >= 32 * 512 * 4 + 32 * 2048 * 6 + 320 * 512 * 6
    assert lib.moe_decode_tokens_workspace_bytes(ctypes.byref(s), 33) == 0
    assert lib.moe_decode_tokens_workspace_bytes(ctypes.byref(s), 0) == 0
    base = dict(shape=ctypes.byref(s), layer=3, T=32, x=FAKE, eps=-1.0, w=FAKE, bias=None, table=FAKE, codebook=FAKE,
                ids=FAKE, weights=FAKE, slots=FAKE, miss=FAKE, ctrl=FAKE, logits=None, y=FAKE, acc=0, ws=FAKE,
                ws_bytes=need, stream=None)
    call = lambda **c: lib.moe_decode_tokens(*_with(base, **c))  # noqa: E731
    for c in (dict(layer=4), dict(layer=-1), dict(T=-1), dict(ws_bytes=need - 1), dict(ws=None), dict(ws=ODD),
              dict(x=ODD), dict(w=ODD), dict(table=None), dict(miss=None), dict(w=None, logits=FAKE),
              *[{k: None} for k in ("x", "codebook", "ids", "weights", "slots", "ctrl", "y")]):
        assert call(**c) == INVALID, c
        assert b"moe_decode_tokens" in lib.rl_last_error()
    assert call(T=33) == UNSUPPORTED
    bad = RlShape.of(384, 512, 10, 512, 4)
    assert call(shape=ctypes.byref(bad)) == UNSUPPORTED
    assert lib.moe_decode_tokens_workspace_bytes(ctypes.byref(bad), 4) == 0
    assert call(T=0, x=None, y=None, ids=None, ws=None, ws_bytes=0) == 0


def test_add_rmsnorm_refusals(lib):
    base = dict(x=FAKE, res=FAKE, gain=FAKE, dtype=2, T=4, H=2048, eps=1e-6, x_out=FAKE, xn=FAKE, q=FAKE, scale=FAKE,
                group=128, stream=None)
    call = lambda **c: lib.rl_add_rmsnorm(*_with(base, **c))  # noqa: E731
    base["xn"] = ctypes.c_void_p(1 << 21)
    for c in (dict(dtype=3), dict(dtype=-1), dict(T=-1), dict(H=0), dict(eps=-1.0), dict(eps=float("nan")),
              dict(x=None), dict(q=None), dict(scale=None), dict(x_out=None, xn=None, q=None, scale=None), dict(H=2080),
              dict(xn=FAKE), *[{k: ODD} for k in ("x", "res", "gain", "x_out", "xn", "q", "scale")]):
        assert call(**c) == INVALID, c
        assert b"rl_add_rmsnorm" in lib.rl_last_error()
    for c in (dict(H=2052), dict(H=16512), dict(group=16), dict(group=256)):
        assert call(**c) == UNSUPPORTED, c
    assert call(T=0, x=None, q=None, scale=None, xn=None, x_out=None) == 0


def test_q4_matvec_refusals(lib):
    base = dict(w=FAKE, ws=FAKE, N=100, K=512, group=64, x=FAKE, xdt=3, xs=FAKE, T=4, y=FAKE, ydt=0, acc=0, stream=None)
    call = lambda **c: lib.rl_q4_matvec(*_with(base, **c))  # noqa: E731
    for c in (dict(xdt=4), dict(xdt=-1), dict(ydt=3), dict(N=0), dict(K=0), dict(T=-1), dict(K=544), dict(w=None),
              dict(ws=None), dict(x=None), dict(y=None), dict(xs=None), dict(xdt=0), dict(w=ODD), dict(ws=ODD),
              dict(x=ODD), dict(xs=ODD), dict(y=ODD)):
        assert call(**c) == INVALID, c
        assert b"rl_q4_matvec" in lib.rl_last_error()
    for c in (dict(group=16), dict(group=256, K=512), dict(K=8256), dict(N=(1 << 26) + 1)):
        assert call(**c) == UNSUPPORTED, c
    assert call(T=0, w=None, ws=None, x=None, xs=None, y=None) == 0


def test_logprobs_refusals(lib):
    need = lib.rl_logprobs_workspace_bytes(16, 100003, 20)
    assert need > 0
    assert lib.rl_logprobs_workspace_bytes(16, 100003, 33) == 0 and lib.rl_logprobs_workspace_bytes(0, 5, 1) == 0
    base = dict(x=FAKE, dtype=1, T=16, V=100003, targets=FAKE, logprob=FAKE, entropy=FAKE, n=20, ids=FAKE, top=FAKE,
                ws=FAKE, ws_bytes=need, stream=None)
    call = lambda **c: lib.rl_logprobs(*_with(base, **c))  # noqa: E731
    odd1 = ctypes.c_void_p((1 << 20) + 1)
    for c in (dict(dtype=3), dict(T=-1), dict(V=0), dict(n=-1), dict(n=20, V=19), dict(x=None), dict(targets=None),
              dict(logprob=None), dict(ids=None), dict(top=None), dict(n=0), dict(ws=None), dict(ws_bytes=need - 1),
              dict(ws=ODD), dict(x=odd1), dict(targets=ODD), dict(entropy=ODD),
              dict(targets=None, logprob=None, entropy=None, n=0, ids=None, top=None)):
        assert call(**c) == INVALID, c
        assert b"rl_logprobs" in lib.rl_last_error()
    for c in (dict(n=33), dict(V=(1 << 30) + 1)):
        assert call(**c) == UNSUPPORTED, c
    assert call(T=0, x=None, targets=None, logprob=None, entropy=None, ids=None, top=None, ws=None, ws_bytes=0) == 0


def test_workspace_is_enough_for_every_split(lib):
    """More rows than one launch takes: the rest may be few rows in more segments."""
    for T in (1, 5, 4096, 4097, 9000):
        for V in (1, 4096, 131072):
            full = lib.rl_logprobs_workspace_bytes(T, V, 32)
            rest = T % 4096 or 4096
            assert full >= lib.rl_logprobs_workspace_bytes(min(rest, T), V, 32)
            assert full >= lib.rl_logprobs_workspace_bytes(min(T, 4096), V, 32)


def test_binding_checks_types_and_sizes():
    """The library sees addresses only: the binding refuses tensors of another type or size."""
    torch = pytest.importorskip("torch")
    from quantized_moe_expert_rl_gb300 import _lib as L
    x = torch.zeros(2, 256)
    with pytest.raises(ValueError, match="x:"):
        L.rl_add_rmsnorm(x.double(), 2, 256, 1e-6, xn=x)
    with pytest.raises(ValueError, match="x:"):
        L.rl_add_rmsnorm(x, 3, 256, 1e-6, xn=x)
    with pytest.raises(ValueError, match="xn:"):
        L.rl_add_rmsnorm(x, 2, 256, 1e-6, xn=x.half())
    with pytest.raises(ValueError, match="gain:"):
        L.rl_add_rmsnorm(x, 2, 256, 1e-6, gain=x[0].half(), xn=x)
    w, ws, y = torch.zeros(5, 128, dtype=torch.uint8), torch.zeros(5, 2).half(), torch.zeros(2, 5)
    with pytest.raises(ValueError, match="w_scale:"):
        L.rl_q4_matvec(w, ws, x, y, 2, 5, 256, 64)
    with pytest.raises(ValueError, match="w:"):
        L.rl_q4_matvec(w[:4], ws, x, y, 2, 5, 256, 128)
    with pytest.raises(ValueError, match="targets:"):
        L.rl_logprobs(x, 2, 256, torch.zeros(2, dtype=torch.int64), y, None, 0, None, None, None, 0)


@pytest.mark.parametrize("what, small", [
    ("x", lambda t: t[:2]), ("y", lambda t: t[:2]), ("x", lambda t: t.half()), ("w_router", lambda t: t[:-1]),
    ("bias", lambda t: t[:-1]), ("residency", lambda t: t[:0]), ("codebook", lambda t: t[:-1]),
    ("ids", lambda t: t[:2]), ("weights", lambda t: t[:2]), ("slots", lambda t: t.int()), ("miss", lambda t: t[:0]),
    ("ctrl", lambda t: t[:1]), ("logits_out", lambda t: t[:2]), ("ws", lambda t: t[:-1])])
def test_binding_checks_the_buffers_of_a_layer(what, small):
    """A step of fewer rows than the buffers' tokens, or any buffer too small for the call, is refused before
    the library sees its address."""
    torch = pytest.importorskip("torch")
    from quantized_moe_expert_rl_gb300 import _lib as L
    sh, T = L.RlShape.of(256, 8, 2, 256, 1), 3
    i32, i64 = torch.int32, torch.int64
    b = dict(x=torch.zeros(T, 256), w_router=torch.zeros(8, 256), bias=torch.zeros(8),
             residency=torch.zeros(1, 8, dtype=i64), codebook=torch.zeros(256, 8, dtype=torch.int8),
             ids=torch.zeros(T, 2, dtype=i32), weights=torch.zeros(T, 2), slots=torch.zeros(T, 2, dtype=i64),
             miss=torch.zeros(1, dtype=i32), ctrl=torch.zeros(2, dtype=i32), logits_out=torch.zeros(T, 8),
             y=torch.zeros(T, 256), ws=torch.zeros(L.moe_decode_tokens_workspace_bytes(sh, T), dtype=torch.uint8))
    size = b["ws"].numel()
    b[what] = small(b[what])
    with pytest.raises(ValueError, match=f"^{what}:"):
        L.moe_decode_tokens(sh, 0, T, b["x"], -1.0, b["w_router"], b["bias"], b["residency"], b["codebook"], b["ids"],
                            b["weights"], b["slots"], b["miss"], b["ctrl"], b["logits_out"], b["y"], 0, b["ws"], size)


def test_binding_checks_the_workspace_of_logprobs():
    torch = pytest.importorskip("torch")
    from quantized_moe_expert_rl_gb300 import _lib as L
    x, size = torch.zeros(2, 256), L.rl_logprobs_workspace_bytes(2, 256, 0)
    with pytest.raises(ValueError, match="^ws:"):
        L.rl_logprobs(x, 2, 256, None, None, torch.zeros(2), 0, None, None,
                      torch.zeros(size - 1, dtype=torch.uint8), size)


@pytest.mark.parametrize("group", [32, 64, 128])
def test_pack_q4(group):
    """Values come back within half a step of their group's scale (rounded to half precision, 2^-11
    relative, times at most 7 steps), zeros as zeros, the byte order as documented."""
    torch = pytest.importorskip("torch")
    from quantized_moe_expert_rl_gb300.engine import pack_q4
    torch.manual_seed(3)
    v = torch.randn(9, 256)
    v[4] = 0
    w, s = pack_q4(v, group)
    assert w.shape == (9, 128) and w.dtype == torch.uint8 and s.shape == (9, 256 // group) and s.dtype == torch.float16
    q = torch.stack((w & 15, w >> 4), 2).view(9, 256).float() - 8
    back = q * s.float().repeat_interleave(group, 1)
    step = s.float().repeat_interleave(group, 1)
    assert torch.all((back - v).abs() <= step * (0.5 + 8 * 2.0 ** -11))
    assert torch.all(back[4] == 0)


@pytest.mark.parametrize("what, dtype", [
    ("x", "int32"), ("w_router", "int32"), ("bias", "int32"), ("residency", "float64"), ("codebook", "bool"),
    ("ids", "float32"), ("weights", "int32"), ("slots", "float64"), ("miss", "float32"), ("ctrl", "float32"),
    ("logits_out", "int32"), ("y", "int32")])
def test_binding_checks_the_types_of_a_layer(what, dtype):
    """A tensor of another type of the same width (ids and weights changed over, say) is refused: the
    library would read its bits as what they are not."""
    torch = pytest.importorskip("torch")
    from quantized_moe_expert_rl_gb300 import _lib as L
    sh, T = L.RlShape.of(256, 8, 2, 256, 1), 3
    i32, i64 = torch.int32, torch.int64
    b = dict(x=torch.zeros(T, 256), w_router=torch.zeros(8, 256), bias=torch.zeros(8),
             residency=torch.zeros(1, 8, dtype=i64), codebook=torch.zeros(256, 8, dtype=torch.int8),
             ids=torch.zeros(T, 2, dtype=i32), weights=torch.zeros(T, 2), slots=torch.zeros(T, 2, dtype=i64),
             miss=torch.zeros(1, dtype=i32), ctrl=torch.zeros(2, dtype=i32), logits_out=torch.zeros(T, 8),
             y=torch.zeros(T, 256), ws=torch.zeros(L.moe_decode_tokens_workspace_bytes(sh, T), dtype=torch.uint8))
    b[what] = b[what].to(getattr(torch, dtype))
    with pytest.raises(ValueError, match=f"^{what}:"):
        L.moe_decode_tokens(sh, 0, T, b["x"], -1.0, b["w_router"], b["bias"], b["residency"], b["codebook"], b["ids"],
                            b["weights"], b["slots"], b["miss"], b["ctrl"], b["logits_out"], b["y"], 0, b["ws"],
                            b["ws"].numel())


@pytest.mark.parametrize("what, dtype", [("targets", "float32"), ("logprob", "int32"), ("entropy", "int32"),
                                         ("top_ids", "float32"), ("top_logprob", "int32")])
def test_binding_checks_the_types_of_logprobs(what, dtype):
    torch = pytest.importorskip("torch")
    from quantized_moe_expert_rl_gb300 import _lib as L
    b = dict(targets=torch.zeros(2, dtype=torch.int32), logprob=torch.zeros(2), entropy=torch.zeros(2),
             top_ids=torch.zeros(2, 3, dtype=torch.int32), top_logprob=torch.zeros(2, 3))
    b[what] = b[what].to(getattr(torch, dtype))
    ws = torch.zeros(L.rl_logprobs_workspace_bytes(2, 256, 3), dtype=torch.uint8)
    with pytest.raises(ValueError, match=f"^{what}:"):
        L.rl_logprobs(torch.zeros(2, 256), 2, 256, b["targets"], b["logprob"], b["entropy"], 3, b["top_ids"],
                      b["top_logprob"], ws, ws.numel())


def test_binding_checks_the_types_of_eight_bits():
    """The 8-bit copy of a norm is e4m3 (or its bytes), not another 8-bit float; 4-bit weights are bytes."""
    torch = pytest.importorskip("torch")
    from quantized_moe_expert_rl_gb300 import _lib as L
    x, scale = torch.zeros(2, 256), torch.zeros(2, 2)
    for dt in (torch.float8_e5m2, torch.bool):
        with pytest.raises(ValueError, match="^q:"):
            L.rl_add_rmsnorm(x, 2, 256, 1e-6, q=torch.zeros(2, 256).to(dt), scale=scale)
    with pytest.raises(ValueError, match="^w:"):
        L.rl_q4_matvec(torch.zeros(5, 128).to(torch.float8_e4m3fn), torch.zeros(5, 2).half(), x, torch.zeros(2, 5), 2, 5,
                       256, 128)
