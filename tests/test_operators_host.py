"""rl_f8_matmul, rl_f8_gated, rl_sample and the drivers that call them, without a GPU: refusals made on the host
before any launch, the packing of 8-bit weights, and the drivers with the library replaced by a stand-in."""
import ctypes
from dataclasses import replace

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import synth  # noqa: E402
from tests._fake_lib import FakeModel  # noqa: E402
from tests.test_tokens_host import StepLib  # noqa: E402

from quantized_moe_expert_rl_gb300._lib import RL_NO_EARLY_OUT  # noqa: E402

INVALID, UNSUPPORTED = 1, 2
FAKE, ODD = ctypes.c_void_p(1 << 20), ctypes.c_void_p((1 << 20) + 2)
W = replace(synth.WORKLOADS["tiny"], n_layers=3)
H, I, V = W.hidden, 48, 53


@pytest.fixture(scope="module")
def lib():
    from quantized_moe_expert_rl_gb300 import _lib, build
    build.build()
    return _lib.load()


def _with(args, **changes):
    return list({**args, **changes}.values())


def test_f8_matmul_refusals(lib):
    base = dict(w=FAKE, ws=FAKE, N=1000, K=2048, x=FAKE, xs=FAKE, T=4, res=FAKE, y=FAKE, dtype=0, layer=0, ctrl=FAKE, stream=None)
    call = lambda **c: lib.rl_f8_matmul(*_with(base, **c))  # noqa: E731
    byte = ctypes.c_void_p((1 << 20) + 8)
    for c in (dict(dtype=3), dict(dtype=-1), dict(T=-1), dict(N=0), dict(K=0), dict(layer=-1), dict(w=byte), dict(x=byte),
              *[{k: ODD} for k in ("w", "ws", "x", "xs", "res", "y", "ctrl")],
              *[{k: None} for k in ("w", "ws", "x", "xs", "y")]):
        assert call(**c) == INVALID, c
        assert b"rl_f8_matmul" in lib.rl_last_error()
    for c in (dict(K=2040), dict(K=8), dict(N=(1 << 26) + 1), dict(T=(1 << 22) + 1), dict(K=(1 << 20) + 16)):
        assert call(**c) == UNSUPPORTED, c
    assert call(T=0, x=None, xs=None, y=None, res=None) == 0


def test_f8_gated_refusals(lib):
    base = dict(wg=FAKE, sg=FAKE, wu=FAKE, su=FAKE, I=512, K=2048, x=FAKE, xs=FAKE, T=4, h=FAKE, dtype=0, q=FAKE, scale=FAKE,
                layer=0, ctrl=FAKE, stream=None)
    call = lambda **c: lib.rl_f8_gated(*_with(base, **c))  # noqa: E731
    for c in (dict(dtype=3), dict(T=-1), dict(I=0), dict(K=-16), dict(layer=-1), dict(h=None, q=None, scale=None), dict(q=None),
              dict(scale=None), *[{k: ODD} for k in ("wg", "sg", "wu", "su", "x", "xs", "h", "q", "scale", "ctrl")],
              *[{k: None} for k in ("wg", "sg", "wu", "su", "x", "xs")]):
        assert call(**c) == INVALID, c
        assert b"rl_f8_gated" in lib.rl_last_error()
    assert call(K=24) == UNSUPPORTED
    assert call(T=0, x=None, xs=None, h=None, q=None, scale=None) == 0


def test_sample_refusals(lib):
    base = dict(x=FAKE, dtype=0, T=4, V=1000, u=FAKE, temperature=FAKE, k=FAKE, p=FAKE, m=FAKE, ids=FAKE, logprob=FAKE, stream=None)
    call = lambda **c: lib.rl_sample(*_with(base, **c))  # noqa: E731
    for c in (dict(dtype=3), dict(dtype=-1), dict(T=-1), dict(V=0), dict(x=None), dict(u=None), dict(ids=None),
              dict(x=ctypes.c_void_p((1 << 20) + 1), dtype=2),
              *[{k: ODD} for k in ("x", "u", "temperature", "k", "p", "m", "ids", "logprob")]):
        assert call(**c) == INVALID, c
        assert b"rl_sample" in lib.rl_last_error()
    for c in (dict(V=(1 << 26) + 1), dict(T=(1 << 24) + 1)):
        assert call(**c) == UNSUPPORTED, c
    assert call(T=0, x=None, u=None, ids=None) == 0


def test_binding_refuses_types_sizes_and_host_tensors():
    """What the library cannot see is refused by the binding, before the library is asked."""
    from quantized_moe_expert_rl_gb300 import _lib as L
    f8, f = torch.float8_e4m3fn, torch.zeros
    w, ws, x, xs, y = f(200, 256).to(f8), f(2, 2), f(3, 256).to(f8), f(3, 2), f(3, 200)
    good = [w, ws, x, xs, y, 3, 200, 256]
    for i, bad in ((0, f(200, 256)), (0, f(100, 256).to(f8)), (1, f(2, 1)), (1, f(2, 2).double()), (2, f(2, 256).to(f8)),
                   (3, f(3, 1)), (4, f(3, 200).double()), (4, f(2, 200)), (5, 4)):
        with pytest.raises(ValueError):
            L.rl_f8_matmul(*[bad if i == j else a for j, a in enumerate(good)])
    with pytest.raises(ValueError, match="res"):
        L.rl_f8_matmul(*good, res=y.half())
    with pytest.raises(ValueError, match="ctrl"):
        L.rl_f8_matmul(*good, ctrl=torch.zeros(1, dtype=torch.int32))
    gated = [w, ws, w, ws, x, xs, 3, 200, 256]
    for kw in (dict(h=f(3, 100)), dict(q=f(3, 200), scale=f(3, 2)), dict(q=f(3, 200).to(f8), scale=f(3, 1))):
        with pytest.raises(ValueError):
            L.rl_f8_gated(*gated, **kw)
    i32 = torch.int32
    for args, kw in (((f(2, 10).double(), 2, 10, f(2), f(2, dtype=i32)), {}), ((f(2, 9), 2, 10, f(2), f(2, dtype=i32)), {}),
                     ((f(2, 10), 2, 10, f(3), f(2, dtype=i32)), {}), ((f(2, 10), 2, 10, f(2), f(2)), {}),
                     ((f(2, 10), 2, 10, f(2), f(2, dtype=i32)), dict(top_k=f(2))),
                     ((f(2, 10), 2, 10, f(2), f(2, dtype=i32)), dict(top_p=f(1)))):
        with pytest.raises(ValueError):
            L.rl_sample(*args, **kw)


@pytest.mark.parametrize("N,K", [(128, 128), (200, 384), (1, 16), (300, 144)])
def test_pack_f8(N, K):
    """Values are off by at most half a step of e4m3 (2^-4 relative; 2^-10 of the scale below its smallest normal), the largest of
    a block is 448 steps, a block of zeros has scale 0."""
    from quantized_moe_expert_rl_gb300 import engine
    w = torch.randn(N, K, generator=torch.Generator().manual_seed(N))
    w[:128, :128] = 0
    q, scale = engine.pack_f8(w)
    assert q.shape == w.shape and q.dtype == torch.float8_e4m3fn and scale.shape == (-(-N // 128), -(-K // 128))
    assert scale[0, 0] == 0 and bool((q[:128, :128].float() == 0).all())
    s = scale.double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    assert torch.all((q.double() * s - w.double()).abs() <= w.double().abs() * (2.0 ** -4 + 2.0 ** -22) + 2.0 ** -10 * 1.001 * s)
    for b in range(scale.shape[0]):
        for c in range(scale.shape[1]):
            block = q[128 * b:128 * b + 128, 128 * c:128 * c + 128].float()
            assert float(block.abs().max()) == (448 if scale[b, c] > 0 else 0)


class OperatorLib(StepLib):
    """StepLib with the 8-bit products and sampling: the shared expert adds 1 to every row of y."""

    def rl_add_rmsnorm(self, x, T, H, eps, res=None, gain=None, x_out=None, xn=None, q=None, scale=None, group=128, stream=None):
        super().rl_add_rmsnorm(x, T, H, eps, res, gain, x_out, xn, q, scale, group, stream)
        self.log.append(("norm", T, x.clone()))

    log = None

    def moe_decode_tokens(self, shape, layer, T, *a, **k):
        self.log.append(("moe", layer))
        super().moe_decode_tokens(shape, layer, T, *a, **k)

    def rl_f8_gated(self, w_gate, gate_scale, w_up, up_scale, x, x_scale, T, I, K, h=None, q=None, scale=None, layer=0, ctrl=None,
                    stream=None):
        assert w_gate.shape == w_up.shape == (I, K) and x.shape == (T, K) and q.shape == (T, I) and scale.shape == (T, -(-I // 128))
        self.log.append(("gated", layer, T))
        if int(ctrl[0]) > layer:
            q.fill_(1.0)

    def rl_f8_matmul(self, w, w_scale, x, x_scale, y, T, N, K, res=None, layer=0, ctrl=None, stream=None):
        assert w.shape == (N, K) and x.shape == (T, K) and y.shape == (T, N)
        self.log.append(("f8", layer, T, N))
        if ctrl is None:
            y.fill_(1.0)
        elif int(ctrl[0]) > layer:
            assert res is y
            y.add_(1.0)

    def rl_sample(self, logits, T, V, uniform, ids, temperature=None, top_k=None, top_p=None, min_p=None, logprob=None, stream=None):
        assert logits.shape == (T, V) and all(t is None or t.numel() == T for t in (uniform, ids, temperature, top_k, top_p, logprob))
        self.log.append(("sample", T))
        ids.copy_(torch.arange(T) % V)

    NAMES = StepLib.NAMES + ("rl_f8_gated", "rl_f8_matmul", "rl_sample")


@pytest.fixture
def env(monkeypatch):
    from quantized_moe_expert_rl_gb300 import engine
    m = FakeModel(W)
    lib = OperatorLib(m)
    lib.log = []
    lib.install(monkeypatch, engine)
    return engine, m, lib


def _shared(engine, T):
    g = torch.Generator().manual_seed(1)
    w = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    first = engine.SharedExpert.make(w(I, H), w(I, H), w(H, I), T)
    return [first] + [engine.SharedExpert.make(w(I, H), w(I, H), w(H, I), T, like=first) for _ in range(W.n_layers - 1)]


def test_shared_expert_reads_the_rows_before_the_routed_ones_add(env):
    engine, m, lib = env
    T = 2
    b = engine.TokensBuffers.make(m, 4)
    x = torch.from_numpy(synth.tokens(W, 0, T))
    plain = torch.empty_like(x)
    engine.enqueue_tokens(m, b, x, plain)
    lib.log.clear()
    m.shared = _shared(engine, 4)
    y = torch.empty_like(x)
    engine.enqueue_tokens(m, b, x, y)
    assert [e[:2] if e[0] != "norm" else e[:1] for e in lib.log] == [
        e for l in range(W.n_layers) for e in (("norm",), ("moe", l), ("gated", l), ("f8", l))]
    assert torch.equal(lib.log[0][2], x)
    one = x.clone()
    m.shared = None
    engine.enqueue_tokens_layer(m, b, 0, one, one, stacked=True)
    m.shared = _shared(engine, 4)
    assert torch.equal(lib.log[4][2], one + 1)  # the second layer's input: the first layer's routed sum and shared expert


def test_shared_expert_waits_for_a_stopped_layer(env):
    """A layer that stops for a fill leaves its shared expert out; it runs with the layer's experts."""
    engine, _, lib = env
    m = FakeModel(replace(W, n_resident=24))
    lib2 = OperatorLib(m)
    lib2.log = lib.log
    mp = pytest.MonkeyPatch()
    lib2.install(mp, engine)
    try:
        b = engine.TokensBuffers.make(m, 3)
        m.shared = _shared(engine, 3)
        x = torch.from_numpy(synth.tokens(W, 0, 3))
        y, yf = torch.empty_like(x), torch.empty_like(x)
        st = engine.run_bounded_tokens(m, b, x, y)
        assert st.early_outs
        b.ctrl.copy_(torch.tensor([RL_NO_EARLY_OUT, 0], dtype=torch.int32))
        engine.enqueue_tokens(m, b, x, yf)  # everything is resident now
        assert torch.equal(y, yf)
    finally:
        mp.undo()


def test_shared_expert_refusals(env):
    engine, m, lib = env
    f = torch.zeros
    with pytest.raises(ValueError, match="expected"):
        engine.SharedExpert.make(f(I, H), f(I, H), f(I, H), 2)
    with pytest.raises(ValueError, match="multiples"):
        engine.SharedExpert.make(f(40, H), f(40, H), f(H, 40), 2)
    first = engine.SharedExpert.make(f(I, H), f(I, H), f(H, I), 2)
    with pytest.raises(ValueError, match="share"):
        engine.SharedExpert.make(f(I, H), f(I, H), f(H, I), 4, like=first)
    b = engine.TokensBuffers.make(m, 4)
    x = torch.from_numpy(synth.tokens(W, 0, 4))
    y = torch.empty_like(x)
    m.shared = _shared(engine, 3)
    with pytest.raises(ValueError, match="buffers hold"):
        engine.enqueue_tokens(m, b, x, y)
    m.shared = m.shared[:2]
    with pytest.raises(ValueError, match="shared experts for"):
        engine.enqueue_tokens(m, b, x, y)
    assert not any(e[0] == "moe" for e in lib.log)
    # paths that run the routed experts only
    for call in (lambda: engine.enqueue_decode_token(m, None, x[0], y[0], True),
                 lambda: engine.enqueue_decode_token_fused(m, None, x[0], y[0]),
                 lambda: engine.run_bounded_decode_token(m, None, x[0], y[0]),
                 lambda: engine.run_bounded_decode_token_device(m, None, x[0], y[0], None)):
        with pytest.raises(ValueError, match="routed experts only"):
            call()


@pytest.mark.parametrize("bits", [4, 8])
def test_generate_rows(env, bits):
    """The head and the sampler get the step's rows; a smaller step their first ones; more rows are refused."""
    engine, m, lib = env
    b = engine.TokensBuffers.make(m, 5)
    head = engine.Head.make(torch.randn(V, H, generator=torch.Generator().manual_seed(2)), 4, top_n=3, bits=bits)
    s = engine.Sampler.make(4, device="cpu", temperature=0.7, top_k=20, top_p=0.9)
    assert s.min_p is None and s.top_k.dtype == torch.int32 and head.bits == bits
    for T in (4, 1, 3):
        lib.log.clear(), lib.rows.clear()
        x = torch.from_numpy(synth.tokens(W, 0, T))
        ids = engine.enqueue_generate(m, b, head, s, x, torch.empty_like(x))
        assert ids.data_ptr() == s.ids.data_ptr() and ids.tolist() == list(range(T))
        assert ("sample", T) in lib.log and (("f8", 0, T, V) in lib.log) == (bits == 8)
        assert ("rl_logprobs", T) in lib.rows and all(n == T for _, n in lib.rows)
    x = torch.from_numpy(synth.tokens(W, 0, 4))
    with pytest.raises(ValueError, match="sampler holds"):
        engine.enqueue_generate(m, b, head, engine.Sampler.make(3, device="cpu"), x, torch.empty_like(x))
    x5 = torch.zeros(5, H)
    with pytest.raises(ValueError, match="head holds"):
        engine.enqueue_generate(m, b, head, s, x5, torch.empty_like(x5))
    with pytest.raises(ValueError, match="sampler holds"):
        engine.enqueue_sample(s, torch.zeros(5, V))


def test_head_refusals(env):
    engine = env[0]
    for kw in (dict(bits=6), dict(bits=8, group=64)):
        with pytest.raises(ValueError, match="bits"):
            engine.Head.make(torch.zeros(V, H), 2, **kw)
    with pytest.raises(ValueError, match="columns"):
        engine.Head.make(torch.zeros(V, 192), 2, bits=8)
    assert np.isfinite(engine.pack_f8(torch.zeros(5, 16))[1].numpy()).all()
