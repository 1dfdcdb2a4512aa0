"""The drivers of a step of a few tokens (engine.enqueue_tokens, enqueue_verify, run_bounded_tokens)
on the CPU, with the C library replaced by a stand-in that follows the header: which rows the layers
and the output head are given, and what the drivers refuse."""
from dataclasses import replace

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import synth  # noqa: E402
from tests._fake_lib import FakeLib, FakeModel, _u64  # noqa: E402
from tests._gpu_common import rel_l2  # noqa: E402

from quantized_moe_expert_rl_gb300._lib import (  # noqa: E402
    RL_DEVERR_MISSING, RL_DEVERR_WAIT_TIMEOUT, RL_NO_EARLY_OUT)

W = replace(synth.WORKLOADS["tiny"], n_layers=4, n_resident=24, zipf_s=1.1)
H, V = W.hidden, 53


class StepLib(FakeLib):
    """The entry points of a step of a few tokens beside those of FakeLib.  rows: (function, T) of
    every call.  device_error: bits that moe_decode_tokens with a given routing raises at a layer,
    leaving y as it was."""

    def __init__(self, model):
        super().__init__(model)
        self.rows, self.device_error = [], {}

    def moe_decode_tokens_workspace_bytes(self, shape, T):
        return 256 + T

    def rl_logprobs_workspace_bytes(self, T, V, top_n):
        return 256

    def moe_decode_tokens(self, shape, layer, T, x, norm_eps, w_router, bias, residency, codebook, ids, weights, slots,
                          miss, ctrl, logits_out, y, accumulate, ws, ws_bytes, stream=None):
        self.rows.append(("moe_decode_tokens", T))
        K = self.w.top_k
        for t, n in ((x, T * H), (ids, T * K), (weights, T * K), (slots, T * K), (y, T * H)):
            assert t.is_contiguous() and t.numel() >= n
        routed = w_router is not None
        if T == 0 or (int(ctrl[0]) < layer if routed else int(ctrl[0]) <= layer):
            return
        row = lambda t, m: t.view(-1)[:T * m].view(T, m)  # noqa: E731
        xn, ids, weights, slots, y = self._xn(row(x, H), norm_eps), row(ids, K), row(weights, K), row(slots, K), row(y, H)
        if routed:
            r = self._route_into(layer, xn, w_router, bias, residency, ids, weights, slots, miss, ctrl, logits_out)
            if r.miss > 0:
                return
        else:
            bits = self.device_error.get(layer, 0) | (RL_DEVERR_MISSING if bool((slots == 0).any()) else 0)
            if bits:
                ctrl[1] = int(ctrl[1]) | bits
                return
        self.runs.append(("moe_decode_tokens", layer))
        out = self._experts(xn, _u64(slots), weights.double().numpy())
        y.copy_(torch.from_numpy(((y.double().numpy() if accumulate else 0.0) + out).astype(np.float32)))

    def rl_add_rmsnorm(self, x, T, H, eps, res=None, gain=None, x_out=None, xn=None, q=None, scale=None, group=128,
                       stream=None):
        self.rows.append(("rl_add_rmsnorm", T))
        assert x.numel() == q.numel() == T * H and scale.numel() == T * (H // group) and q.is_contiguous()
        self.normed = x.clone()
        q.copy_(torch.ones(T, H).to(q.dtype))

    def rl_q4_matvec(self, w, w_scale, x, y, T, N, K, group, x_scale=None, accumulate=0, stream=None):
        self.rows.append(("rl_q4_matvec", T))
        assert x.numel() == T * K and y.numel() == T * N and x_scale.numel() == T * (K // group) and y.is_contiguous()
        y.fill_(1.0)

    def rl_logprobs(self, logits, T, V, targets, logprob, entropy, top_n, top_ids, top_logprob, ws, ws_bytes,
                    stream=None):
        self.rows.append(("rl_logprobs", T))
        assert logits.numel() == T * V and targets.numel() == logprob.numel() == entropy.numel() == T
        assert top_n == 0 or top_ids.numel() == top_logprob.numel() == T * top_n
        logprob.fill_(-1.0)
        if top_n:
            top_ids.fill_(3)

    NAMES = FakeLib.NAMES + ("moe_decode_tokens_workspace_bytes", "moe_decode_tokens", "rl_add_rmsnorm", "rl_q4_matvec",
                             "rl_logprobs_workspace_bytes", "rl_logprobs")


@pytest.fixture
def host(monkeypatch):
    from quantized_moe_expert_rl_gb300 import engine

    def make(w=W):
        m = FakeModel(w)
        lib = StepLib(m)
        lib.install(monkeypatch, engine)
        return engine, m, lib
    return make


def tokens(T, at=0):
    return torch.from_numpy(synth.tokens(W, at, T)).clone()


def a_head(engine, T, top_n=2):
    return engine.Head.make(torch.randn(V, H, generator=torch.Generator().manual_seed(1)), T, group=64, top_n=top_n)


# ---- rows that do not belong together -----------------------------------------------------
def test_more_rows_than_the_buffers_hold_are_refused(host):
    """Every driver, before it launches or writes anything: rows 4 to 7 would come back without a layer."""
    engine, m, lib = host()
    b, head = engine.TokensBuffers.make(m, 4), a_head(engine, 8)
    x, y, t = tokens(8), torch.full((8, H), 7.0), torch.zeros(8, dtype=torch.int32)
    calls = (lambda: engine.enqueue_tokens_layer(m, b, 0, x, y, stacked=False),
             lambda: engine.enqueue_tokens_layer(m, b, 0, x, y, stacked=False, routed=False),
             lambda: engine.enqueue_tokens(m, b, x, y), lambda: engine.run_bounded_tokens(m, b, x, y),
             lambda: engine.enqueue_verify(m, b, head, x, y, t))
    for call in calls:
        with pytest.raises(ValueError, match="8 tokens"):
            call()
    assert lib.rows == [] and torch.all(y == 7.0)


@pytest.mark.parametrize("rows_x, rows_y", [(4, 3), (3, 4), (1, 4), (4, 5)])
def test_input_and_output_of_other_sizes_are_refused(host, rows_x, rows_y):
    """In particular one input row is not spread over all rows of the output."""
    engine, m, lib = host()
    b, head = engine.TokensBuffers.make(m, 4), a_head(engine, 4)
    x, y = tokens(rows_x), torch.full((rows_y, H), 7.0)
    for call in (lambda: engine.enqueue_tokens_layer(m, b, 0, x, y, stacked=False),
                 lambda: engine.enqueue_tokens(m, b, x, y), lambda: engine.run_bounded_tokens(m, b, x, y),
                 lambda: engine.enqueue_verify(m, b, head, x, y, torch.zeros(rows_x, dtype=torch.int32))):
        with pytest.raises(ValueError, match="shape|tokens"):
            call()
    assert lib.rows == [] and torch.all(y == 7.0)


def test_other_widths_and_ranks_are_refused(host):
    engine, m, lib = host()
    b = engine.TokensBuffers.make(m, 2)
    for bad in (torch.zeros(2, H + 8), torch.zeros(2 * H), torch.zeros(2, 1, H)):
        with pytest.raises(ValueError, match="shape"):
            engine.enqueue_tokens(m, b, bad, torch.zeros_like(bad))
    assert lib.rows == []


def test_a_head_or_targets_of_other_sizes_are_refused_before_the_layers_run(host):
    engine, m, lib = host()
    b, x, y = engine.TokensBuffers.make(m, 4), tokens(4), torch.full((4, H), 7.0)
    t = torch.zeros(4, dtype=torch.int32)
    for head, targets in ((a_head(engine, 3), t), (a_head(engine, 4), t[:3]), (a_head(engine, 4), torch.zeros(5, dtype=torch.int32)),
                          (a_head(engine, 4), t.long())):
        with pytest.raises(ValueError):
            engine.enqueue_verify(m, b, head, x, y, targets)
    assert lib.rows == [] and torch.all(y == 7.0)


def test_a_step_as_large_as_its_buffers_runs(host):
    engine, m, lib = host(replace(W, n_resident=-1))
    b, head, x = engine.TokensBuffers.make(m, 4), a_head(engine, 4), tokens(4)
    y, t = torch.empty(4, H), torch.zeros(4, dtype=torch.int32)
    engine.enqueue_verify(m, b, head, x, y, t)
    assert lib.rows == m.L * [("moe_decode_tokens", 4)] + [(f, 4) for f in ("rl_add_rmsnorm", "rl_q4_matvec", "rl_logprobs")]
    assert torch.equal(lib.normed, y) and not torch.equal(y, x)
    z = x.clone()
    engine.enqueue_tokens(m, b, z, z)          # in place
    assert torch.equal(z, y)


# ---- steps of fewer tokens than the buffers hold ------------------------------------------
@pytest.mark.parametrize("T", [0, 1, 3])
def test_a_smaller_step_runs_in_the_same_buffers(host, T):
    """Only its rows are run and written; the results are those of buffers of its own size."""
    engine, m, lib = host(replace(W, n_resident=-1))
    b, head = engine.TokensBuffers.make(m, 5), a_head(engine, 5)
    engine.enqueue_verify(m, b, head, tokens(5), torch.empty(5, H), torch.zeros(5, dtype=torch.int32))
    x, y = tokens(T, at=7), torch.empty(T, H)
    ids, weights = b.ids.clone(), b.weights.clone()
    for out in (head.logits, head.logprob, head.entropy, head.top_logprob, head.top_ids):
        out.fill_(7)
    lib.rows.clear()
    engine.enqueue_verify(m, b, head, x, y, torch.zeros(T, dtype=torch.int32))
    assert {n for _, n in lib.rows} == {T}
    assert torch.all(head.logits[:T] == 1) and torch.all(head.logits[T:] == 7)
    assert torch.all(head.logprob[:T] == -1) and torch.all(head.logprob[T:] == 7)
    assert torch.all(head.top_ids[:T] == 3) and torch.all(head.top_ids[T:] == 7)
    assert torch.equal(b.ids[:, T:], ids[:, T:]) and torch.equal(b.weights[:, T:], weights[:, T:])
    if T:
        own = engine.TokensBuffers.make(m, T)
        z = torch.empty(T, H)
        engine.enqueue_tokens(m, own, x, z)
        assert torch.equal(z, y) and torch.equal(own.ids, b.ids[:, :T]) and torch.equal(own.slots, b.slots[:, :T])


def test_a_smaller_bounded_step_fills_for_its_own_rows_only(host):
    """The rows behind it hold the ids and absent slots of an earlier, larger step."""
    engine, m, lib = host()
    b = engine.TokensBuffers.make(m, 5)
    engine.enqueue_tokens(m, b, tokens(5), torch.empty(5, H))          # stops at a layer; its slots stay absent
    assert bool((b.slots[:, 2:] == 0).any())
    x, y = tokens(2, at=11), torch.empty(2, H)
    st = engine.run_bounded_tokens(m, b, x, y)
    engine2, m2, _ = host()
    b2, y2 = engine2.TokensBuffers.make(m2, 2), torch.empty(2, H)
    st2 = engine2.run_bounded_tokens(m2, b2, x, y2)
    assert (st.early_outs, st.filled, st.fill_bytes) == (st2.early_outs, st2.filled, st2.fill_bytes) and st.filled
    assert torch.equal(y, y2) and np.array_equal(m.table_host, m2.table_host)
    full, mf, libf = host(replace(W, n_resident=-1))
    yf = torch.empty(2, H)
    full.enqueue_tokens(mf, full.TokensBuffers.make(mf, 2), x, yf)
    assert rel_l2(y.numpy(), yf.numpy()) == 0


# ---- error bits of the last launch --------------------------------------------------------
@pytest.mark.parametrize("bits", [RL_DEVERR_MISSING, RL_DEVERR_WAIT_TIMEOUT])
@pytest.mark.parametrize("last", [True, False])
def test_error_bits_after_a_fill_are_raised(host, bits, last):
    """A layer that runs with the routing it was given after a fill and raises an error bit leaves y
    without that layer's experts: an error at the last layer too, after which no launch follows."""
    engine, m, lib = host()
    x, y = tokens(3), torch.empty(3, H)
    stops = engine.run_bounded_tokens(m, engine.TokensBuffers.make(m, 3), x, y).early_outs
    assert stops[-1] == m.L - 1 and len(stops) > 1
    engine, m, lib = host()
    lib.device_error = {stops[-1] if last else stops[0]: bits}
    b = engine.TokensBuffers.make(m, 3)
    with pytest.raises(RuntimeError, match=f"error bits {bits:#x}"):
        engine.run_bounded_tokens(m, b, x, y)
    # the next step on the same buffers starts afresh
    lib.device_error = {}
    engine.run_bounded_tokens(m, b, x, y)
    assert b.ctrl.tolist() == [RL_NO_EARLY_OUT, 0]


@pytest.mark.parametrize("last", [True, False])
@pytest.mark.parametrize("lookahead", [True, False])
def test_error_bits_after_a_fill_are_raised_for_one_token(host, monkeypatch, last, lookahead):
    """The same in run_bounded_decode_token, whose stopped layer runs through moe_decode."""
    engine, m, lib = host()
    x, y = tokens(1, at=2)[0], torch.empty(H)
    stops = engine.run_bounded_decode_token(m, engine.DecodeBuffers.make(m), x, y, lookahead=lookahead).early_outs
    at = stops[-1] if last else stops[0]
    assert not last or at == m.L - 1
    engine, m, lib = host()
    b = engine.DecodeBuffers.make(m)
    real = lib.moe_decode

    def failing(shape, layer, x, norm_eps, slots, weights, codebook, y, accumulate, ctrl, ws, ws_bytes, stream=None):
        if layer == at:
            ctrl[1] = int(ctrl[1]) | RL_DEVERR_MISSING
        else:
            real(shape, layer, x, norm_eps, slots, weights, codebook, y, accumulate, ctrl, ws, ws_bytes)
    monkeypatch.setattr(engine.L, "moe_decode", failing)
    with pytest.raises(RuntimeError, match="device error bits 0x8"):
        engine.run_bounded_decode_token(m, b, x, y, lookahead=lookahead)
