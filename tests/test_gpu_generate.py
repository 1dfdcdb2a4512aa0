"""The operators together, as a program runs them: shared experts beside the routed ones, an output head in 8 bits and the draw
of the next tokens, in the drivers of engine.py."""
from dataclasses import replace

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import synth  # noqa: E402
from tests._gpu_common import REL_F32, REL_TC, rel_l2  # noqa: E402
from tests.test_gpu_sample import NEAR, define  # noqa: E402

TINY = synth.WORKLOADS["tiny"]
NO_EARLY_OUT = 0x7FFFFFFF


@pytest.fixture(scope="module")
def engine():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from quantized_moe_expert_rl_gb300 import build, engine
    build.build()
    return engine


def randn(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).cuda()


def shared_experts(engine, w, T, inter=144):
    H = w.hidden
    out = []
    for l in range(w.n_layers):
        a, b, c = (0.05 * randn(*s, seed=100 + 3 * l + i) for i, s in enumerate(((inter, H), (inter, H), (H, inter))))
        out.append(engine.SharedExpert.make(a, b, c, T, like=out[0] if out else None))
    return out


def weights(pair):
    w, s = pair
    N, K = w.shape
    return w.double() * s.double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]


def shared_ref(e, T):
    """The shared expert in 64 bits from the 8-bit rows it read and the 8-bit hidden rows it wrote: (hidden, output)."""
    x = e.q[:T].double() * e.q_scale[:T].double().repeat_interleave(128, 1)
    a, b = x @ weights(e.gate).t(), x @ weights(e.up).t()
    h = e.h[:T].double() * e.h_scale[:T].double().repeat_interleave(128, 1)[:, :e.h.shape[1]]
    return a * torch.sigmoid(a) * b, h @ weights(e.down).t()


@pytest.mark.parametrize("T", [1, 5, 32])
def test_tokens_with_shared_experts(engine, T):
    """One layer: y = x + MoE(RMSNorm(x)) + shared(RMSNorm(x)), the parts from the same calls made apart."""
    w = replace(TINY, n_layers=1)
    m = engine.Model(w)
    b = engine.TokensBuffers.make(m, 32)
    x = torch.from_numpy(synth.tokens(replace(w, seed=T), 0, T)).cuda()
    plain, y = torch.empty_like(x), torch.empty_like(x)
    engine.enqueue_tokens(m, b, x, plain)
    m.shared = shared_experts(engine, w, 32)
    engine.enqueue_tokens(m, b, x, y)
    torch.cuda.synchronize()
    assert b.ctrl.tolist() == [NO_EARLY_OUT, 0]
    e = m.shared[0]
    hid, out = shared_ref(e, T)
    norm = x.double() / (x.double().square().mean(1, keepdim=True) + 1e-6).sqrt()
    assert rel_l2((e.q[:T].double() * e.q_scale[:T].double().repeat_interleave(128, 1)).cpu().numpy(), norm.cpu().numpy()) <= 2.0 ** -4
    h = e.h[:T].double() * e.h_scale[:T].double().repeat_interleave(128, 1)[:, :e.h.shape[1]]
    assert rel_l2(h.cpu().numpy(), hid.cpu().numpy()) <= 2.0 ** -4
    assert float(out.norm()) > 0.01 * float(plain.double().norm())
    # one f32 rounding of the residual sum beside the product's own error
    assert rel_l2(y.double().cpu().numpy(), (plain.double() + out).cpu().numpy()) <= REL_F32


def test_bounded_tokens_with_shared_experts(engine):
    """A layer that stops for a fill leaves its shared expert out until its experts run: the bits of full residency."""
    w = replace(TINY, n_layers=4, n_resident=24)
    m, full = engine.Model(w), engine.Model(replace(w, n_resident=-1))
    m.shared = full.shared = shared_experts(engine, w, 5)
    b, bf = engine.TokensBuffers.make(m, 5), engine.TokensBuffers.make(full, 5)
    stops = 0
    for step in range(2):
        x = torch.from_numpy(synth.tokens(replace(w, seed=60 + step), 0, 5)).cuda()
        y, yf = torch.empty_like(x), torch.empty_like(x)
        st = engine.run_bounded_tokens(m, b, x, y)
        engine.enqueue_tokens(full, bf, x, yf)
        torch.cuda.synchronize()
        stops += len(st.early_outs)
        assert torch.equal(y, yf) and b.ctrl[1] == 0
    assert stops


@pytest.mark.parametrize("T", [7, 300])
def test_prefill_chunk_with_shared_experts(engine, T):
    """A chunk through every layer with stops and fills, against the chunk with everything resident; one layer against its
    parts."""
    w = replace(TINY, n_layers=3, n_resident=24, tokens=T)
    m, full = engine.Model(w), engine.Model(replace(w, n_resident=-1))
    m.shared = full.shared = shared_experts(engine, w, T)
    pb, pf = engine.PrefillBuffers.make(m, T), engine.PrefillBuffers.make(full, T)
    x = torch.from_numpy(synth.tokens(w, 0, T)).cuda()
    a, c, dev = x.clone(), x.clone(), x.clone()
    st = engine.run_bounded_chunk(m, pb, a)
    engine.run_bounded_chunk(full, pf, c)
    assert st.early_outs and torch.equal(a, c)
    m.reset_residency()
    engine.run_bounded_chunk_device(m, pb, dev)
    assert torch.equal(dev, c)
    one, plain = x.clone(), x.clone()
    engine.enqueue_prefill_route(full, pf, 0, one, True)
    engine.enqueue_prefill_experts(full, pf, 0, one, one, True)
    _, out = shared_ref(full.shared[0], T)
    full.shared = None
    engine.enqueue_prefill_route(full, pf, 0, plain, True)
    engine.enqueue_prefill_experts(full, pf, 0, plain, plain, True)
    assert rel_l2(one.double().cpu().numpy(), (plain.double() + out).cpu().numpy()) <= REL_TC


@pytest.mark.parametrize("bits", [4, 8])
def test_generate_step(engine, bits):
    """Layers with shared experts, norm, head, draw and log probabilities as one step, eager and as a captured graph replayed
    on new tokens and new random numbers."""
    w = replace(TINY, n_layers=2)
    m = engine.Model(w)
    T, V, n = 6, 5003, 4
    m.shared = shared_experts(engine, w, 8)
    b = engine.TokensBuffers.make(m, 8)
    head = engine.Head.make(0.2 * randn(V, w.hidden, seed=32), 8, gain=1 + 0.1 * randn(w.hidden, seed=31), top_n=n, bits=bits)
    s = engine.Sampler.make(8, temperature=0.8, top_k=40, top_p=0.9, min_p=0.01)
    x, y = torch.empty(T, w.hidden, device="cuda"), torch.empty(T, w.hidden, device="cuda")
    graph, seen = None, []
    for step in range(4):
        x.copy_(torch.from_numpy(synth.tokens(replace(w, seed=step), 0, T)))
        s.uniform.copy_(torch.rand(8, generator=torch.Generator().manual_seed(step)))
        if step == 0:
            engine.enqueue_generate(m, b, head, s, x, y)
        elif graph is None:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                engine.enqueue_generate(m, b, head, s, x, y)
            graph.replay()
        else:
            graph.replay()
        torch.cuda.synchronize()
        assert b.ctrl.tolist() == [NO_EARLY_OUT, 0]
        if bits == 8:
            q = head.q[:T].double() * head.q_scale[:T].double().repeat_interleave(128, 1)
            want = q @ weights((head.w, head.scale)).t()
            assert rel_l2(head.logits[:T].cpu().numpy(), want.cpu().numpy()) <= REL_F32
        for t in range(T):
            tok, lp, err, near = define(head.logits[t], float(s.uniform[t]), float(s.temperature[t]), 40,
                                        float(s.top_p[t]), float(s.min_p[t]))
            if near >= NEAR:
                assert int(s.ids[t]) == tok and abs(float(s.logprob[t]) - lp) <= err
        own = torch.log_softmax(head.logits[:T].double(), 1).gather(1, s.ids[:T].long()[:, None])[:, 0]
        assert np.allclose(head.logprob[:T].double().cpu().numpy(), own.cpu().numpy(), atol=2e-6)
        seen.append(s.ids[:T].tolist())
    assert len({tuple(v) for v in seen}) > 1 and s.ids[T:].tolist() == [0, 0]
