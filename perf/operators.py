"""The operators of a small batch of tokens: what is timed, on which inputs, and the plain form of each.

Four operators that a program verifying a few drafted tokens (or decoding a few sequences side by
side) calls one after the other:

  norm   residual addition and RMSNorm, with the normalised row also in 8 bits and group scales
  q4     products of 4-bit weights with group scales and a few activation rows
  moe    a whole routed mixture-of-experts layer (router, experts, combine) for a few tokens
  logp   log probability of given tokens, entropy and the most probable alternatives

`run` computes the plain form with elementary torch operations where `own` is false, and calls the
framework where it is true.  The sizes are those of the framework's workloads (hidden 2048, 512
experts, top-10, intermediate 512) with vocabularies of a generic size.
"""
import math

import numpy as np
import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
F8 = torch.float8_e4m3fn
F8_MAX = 448.0
EPS = 1e-6
BLOCK, BLOCK_BYTES = 256, 66


def listed():
    return [
        # the norm in front of the output head for one decoded token
        dict(name="norm 1 token f32", op="norm", T=1, H=2048, dtype="f32", res=True, gain=True, group=128),
        # the same over a prompt chunk of a 16-bit residual stream
        dict(name="norm 2048 tokens bf16", op="norm", T=2048, H=2048, dtype="bf16", res=True, gain=True, group=128),
        # a shared expert's gate projection for one token: a small matrix, latency
        dict(name="q4 512x2048 1 token", op="q4", N=512, K=2048, T=1, x="f8", y="f32", group=128),
        # a shared expert's down projection for a handful of drafted tokens
        dict(name="q4 2048x512 5 tokens", op="q4", N=2048, K=512, T=5, x="f32", y="f32", group=64),
        # the output head of one token: the largest matrix a decode step reads
        dict(name="q4 head 1 token", op="q4", N=131072, K=2048, T=1, x="f8", y="f32", group=128),
        # an output head of odd height for sixteen sequences, finer groups
        dict(name="q4 odd head 16 tokens", op="q4", N=100003, K=2048, T=16, x="bf16", y="f32", group=32),
        # one decode token through one layer
        dict(name="moe 1 token", op="moe", T=1, H=2048, E=512, K=10, I=512, alike=False, norm=True),
        # drafted tokens of one sequence: they share many of their experts
        dict(name="moe 5 drafted tokens", op="moe", T=5, H=2048, E=512, K=10, I=512, alike=True, norm=True),
        # thirty-two sequences decoded side by side: almost every selection is another expert
        dict(name="moe 32 tokens", op="moe", T=32, H=2048, E=512, K=10, I=512, alike=False, norm=True),
        # the last step of a verified token
        dict(name="logp 1 token", op="logp", T=1, V=131072, dtype="f32", n=20),
        # sixteen sequences, 16-bit logits (exact ties), odd vocabulary
        dict(name="logp 16 tokens bf16", op="logp", T=16, V=100003, dtype="bf16", n=5),
        # the log probabilities of a whole prompt chunk
        dict(name="logp 512 tokens", op="logp", T=512, V=131072, dtype="f32", n=20),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "q4", "moe", "logp"])
    if op == "norm":
        group = rng.choice([32, 64, 128])
        H = 128 * _log(rng, 2, 32)
        return dict(op=op, T=min(_log(rng, 1, 2048), 2048 * 2048 // H), H=H, dtype=rng.choice(["f32", "f16", "bf16"]),
                    res=rng.random() < 0.7, gain=rng.random() < 0.7, group=group)
    if op == "q4":
        K = 128 * _log(rng, 1, 32)
        N = min(_log(rng, 33, 131072), 131072 * 2048 // K)
        T = _log(rng, 1, max(1, min(64, 16 * 100003 * 2048 // (N * K))))
        return dict(op=op, N=N, K=K, T=T, x=rng.choice(["f8", "f32", "f16", "bf16"]),
                    y=rng.choice(["f32", "f32", "bf16"]), group=rng.choice([32, 64, 128]))
    if op == "moe":
        H, I = rng.choice([512, 1024, 2048]), rng.choice([128, 256, 512])
        E = _log(rng, 24, 512)
        return dict(op=op, T=_log(rng, 1, 32), H=H, E=E, K=rng.randint(1, 10), I=I, alike=rng.random() < 0.5,
                    norm=rng.random() < 0.7)
    return dict(op=op, T=_log(rng, 1, 512), V=_log(rng, 1000, 131072), dtype=rng.choice(["f32", "f16", "bf16"]),
                n=rng.choice([0, 1, 5, 20]))


def _record_bytes(c):
    return 3 * c["H"] * c["I"] // BLOCK * BLOCK_BYTES


def work(c):
    """Bytes and operations that no form of the operator can do without."""
    if c["op"] == "norm":
        T, H, b = c["T"], c["H"], DT[c["dtype"]].itemsize
        read = T * H * b * (2 if c["res"] else 1) + (4 * H if c["gain"] else 0)
        write = T * H * b * (2 if c["res"] else 1) + T * H + T * (H // c["group"]) * 4
        return {"bytes": read + write, "flops": 6.0 * T * H}
    if c["op"] == "q4":
        N, K, T = c["N"], c["K"], c["T"]
        xb = 1 + 4 / c["group"] if c["x"] == "f8" else DT[c["x"]].itemsize
        return {"bytes": N * K / 2 + N * (K // c["group"]) * 2 + T * K * xb + T * N * DT[c["y"]].itemsize,
                "flops": 2.0 * T * N * K}
    if c["op"] == "moe":
        T, H, E, K, I = c["T"], c["H"], c["E"], c["K"], c["I"]
        # distinct experts: expected for independent tokens; drafted tokens share at least K
        distinct = K if c["alike"] else E * (1 - (1 - K / E) ** T)
        return {"bytes": E * H * 4 + distinct * _record_bytes(c) + 2 * T * H * 4 + 2048,
                "flops": 2.0 * T * E * H + 6.0 * T * K * H * I}
    T, V, n = c["T"], c["V"], c["n"]
    return {"bytes": T * V * DT[c["dtype"]].itemsize + T * (12 + 8 * n), "flops": 5.0 * T * V}


# ---- inputs -------------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 13)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _randbytes(g, n):
    return torch.randint(-2 ** 31, 2 ** 31 - 1, (-(-n // 4),), generator=g, device="cuda",
                         dtype=torch.int32).view(torch.uint8)[:n]


def prepare(c, seed):
    g, s = _gen(seed), {"c": c}
    empty = lambda *shape, dtype=torch.float32: torch.empty(*shape, dtype=dtype, device="cuda")  # noqa: E731
    if c["op"] == "norm":
        T, H, dt = c["T"], c["H"], DT[c["dtype"]]
        # a residual stream: unit scale with a few strong channels, and a layer's smaller output
        loud = 1 + 15 * (torch.rand(H, generator=g, device="cuda") < 0.01)
        s["x"] = (_randn(g, T, H) * loud).to(dt)
        s["res"] = (0.3 * _randn(g, T, H)).to(dt) if c["res"] else None
        s["gain"] = 1 + 0.2 * _randn(g, H) if c["gain"] else None
        s["x_out"] = empty(T, H, dtype=dt) if c["res"] else None
        s["xn"], s["q"] = empty(T, H, dtype=dt), empty(T, H, dtype=F8)
        s["scale"] = empty(T, H // c["group"])
    elif c["op"] == "q4":
        N, K, T, G = c["N"], c["K"], c["T"], c["group"]
        s["w"] = _randbytes(g, N * K // 2).view(N, K // 2)
        s["ws"] = (0.002 + 0.008 * torch.rand(N, K // G, generator=g, device="cuda")).half()
        x = _randn(g, T, K) * (1 + 15 * (torch.rand(K, generator=g, device="cuda") < 0.01))
        s["xs"] = None
        if c["x"] == "f8":
            s["xs"] = x.view(T, K // G, G).abs().amax(2).clamp_min(1e-20) / F8_MAX
            s["x"] = (x.view(T, K // G, G) / s["xs"][:, :, None]).clamp(-F8_MAX, F8_MAX).view(T, K).to(F8)
        else:
            s["x"] = x.to(DT[c["x"]])
        s["y"] = empty(T, N, dtype=DT[c["y"]])
    elif c["op"] == "moe":
        T, H, E, K, I = c["T"], c["H"], c["E"], c["K"], c["I"]
        rb = _record_bytes(c)
        s["pool"] = _randbytes(g, E * rb).view(E, rb)
        blocks = s["pool"].view(-1, BLOCK_BYTES)
        d = (1e-3 + 3e-3 * torch.rand(blocks.shape[0], generator=g, device="cuda")).half()
        blocks[:, :2] = d.view(torch.uint8).view(-1, 2)
        levels = torch.tensor([8, 25, 43], dtype=torch.int8, device="cuda")
        s["codebook"] = levels[torch.randint(0, 3, (256, 8), generator=g, device="cuda")]
        s["router"] = 0.02 * _randn(g, E, H)
        x = _randn(g, T, H)
        s["x"] = 0.9 * x[:1] + 0.43 * x if c["alike"] else x
        s["base"] = s["pool"].data_ptr()
        s["table"] = s["base"] + rb * torch.arange(E, device="cuda", dtype=torch.int64).view(1, E)
        s["ids"] = empty(T, K, dtype=torch.int32)
        s["weights"] = empty(T, K)
        s["slots"] = empty(T, K, dtype=torch.int64)
        s["miss"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        s["ctrl"] = torch.tensor([0x7FFFFFFF, 0], dtype=torch.int32, device="cuda")
        s["y"] = empty(T, H)
        if own:
            import quantized_moe_expert_rl_gb300 as rl
            s["shape"] = rl.RlShape.of(H, E, K, I, 1)
            s["scratch"] = torch.zeros(rl.moe_decode_tokens_workspace_bytes(s["shape"], T), dtype=torch.uint8,
                                       device="cuda")
    else:
        T, V, n = c["T"], c["V"], c["n"]
        # next-token logits: a broad background and a few likely candidates
        x = 2.0 * _randn(g, T, V) - 4
        likely = torch.randint(0, V, (T, 12), generator=g, device="cuda")
        x.scatter_(1, likely, 9 + 3 * _randn(g, T, 12))
        s["x"] = x.to(DT[c["dtype"]])
        s["targets"] = torch.where(torch.rand(T, generator=g, device="cuda") < 0.7, likely[:, 0],
                                   torch.randint(0, V, (T,), generator=g, device="cuda")).to(torch.int32)
        s["logprob"], s["entropy"] = empty(T), empty(T)
        s["top_ids"] = empty(T, n, dtype=torch.int32) if n else None
        s["top_logprob"] = empty(T, n) if n else None
        if own:
            import quantized_moe_expert_rl_gb300 as rl
            s["scratch"] = torch.zeros(max(16, rl.rl_logprobs_workspace_bytes(T, V, n)), dtype=torch.uint8,
                                       device="cuda")
    return s


# ---- the operators ------------------------------------------------------------------------
def run(s):
    return {"norm": _norm, "q4": _q4, "moe": _moe, "logp": _logp}[s["c"]["op"]](s)


def _norm(s):
    c = s["c"]
    T, H, G = c["T"], c["H"], c["group"]
    if own:
        import quantized_moe_expert_rl_gb300 as rl
        rl.rl_add_rmsnorm(s["x"], T, H, EPS, res=s["res"], gain=s["gain"], x_out=s["x_out"], xn=s["xn"], q=s["q"],
                          scale=s["scale"], group=G)
        return {k: s[k] for k in ("x_out", "xn", "q", "scale")}
    x, dt = s["x"], DT[c["dtype"]]
    if c["res"]:
        x = (x.float() + s["res"].float()).to(dt)
    v = x.float()
    v = v * torch.rsqrt(v.square().mean(1, keepdim=True) + EPS)
    if c["gain"]:
        v = v * s["gain"]
    u = v.view(T, H // G, G)
    scale = u.abs().amax(2) / F8_MAX
    q = torch.where(scale[:, :, None] > 0, u / scale[:, :, None], torch.zeros_like(u)).clamp(-F8_MAX, F8_MAX)
    return {"x_out": x if c["res"] else None, "xn": v.to(dt), "q": q.view(T, H).to(F8), "scale": scale}


def _q4(s):
    c = s["c"]
    N, K, T, G = c["N"], c["K"], c["T"], c["group"]
    if own:
        import quantized_moe_expert_rl_gb300 as rl
        rl.rl_q4_matvec(s["w"], s["ws"], s["x"], s["y"], T, N, K, G, x_scale=s["xs"])
        return s["y"]
    w = s["w"]
    q = torch.stack((w & 15, w >> 4), 2).view(N, K // G, G).float() - 8
    w = (q * s["ws"].float()[:, :, None]).view(N, K)
    x = s["x"].float()
    if s["xs"] is not None:
        x = (x.view(T, K // G, G) * s["xs"][:, :, None]).view(T, K)
    return (x @ w.t()).to(DT[c["y"]])


def _values(records, codebook):
    """Records of 66-byte blocks (fp16 scale, 32 x (codebook row, sign bits)) as f32 values [n][values]."""
    n = records.shape[0]
    b = records.view(n, -1, BLOCK_BYTES)
    d = b[:, :, :2].contiguous().view(torch.float16).float()
    pairs = b[:, :, 2:].reshape(n, -1, 32, 2)
    v = codebook.float()[pairs[..., 0].long()]
    bit = torch.arange(8, device=records.device, dtype=torch.uint8)
    v = v * (1 - 2 * ((pairs[..., 1][..., None] >> bit) & 1).float())
    return (v * d[..., None]).view(n, -1)


def _moe(s):
    c = s["c"]
    T, H, E, K, I = c["T"], c["H"], c["E"], c["K"], c["I"]
    if own:
        import quantized_moe_expert_rl_gb300 as rl
        rl.moe_decode_tokens(s["shape"], 0, T, s["x"], EPS if c["norm"] else -1.0, s["router"], None, s["table"],
                             s["codebook"], s["ids"], s["weights"], s["slots"], s["miss"], s["ctrl"], None, s["y"], 0,
                             s["scratch"], s["scratch"].numel())
        return {"y": s["y"], "ids": s["ids"], "weights": s["weights"]}
    x = s["x"]
    if c["norm"]:
        x = x * torch.rsqrt(x.square().mean(1, keepdim=True) + EPS)
    # in 64 bits: two logits next to each other decide which expert runs
    logits, order = torch.sort((x.double() @ s["router"].double().t()).float(), dim=1, descending=True, stable=True)
    ids = order[:, :K]
    weights = torch.softmax(logits[:, :K], 1)
    slots = s["table"][0][ids]
    rows, inverse = torch.unique((slots - s["base"]) // _record_bytes(c), return_inverse=True)
    w = _values(s["pool"][rows], s["codebook"])
    gate, up = w[:, :2 * H * I].view(-1, 2, I, H).unbind(1)
    down = w[:, 2 * H * I:].view(-1, H, I)
    a, b = gate @ x.t(), up @ x.t()                       # [experts][I][T]
    o = down @ (a * torch.sigmoid(a) * b)                 # [experts][H][T]
    t = torch.arange(T, device=x.device)[:, None]
    y = (o[inverse, :, t.expand(T, K)] * weights[:, :, None]).sum(1)
    return {"y": y, "ids": ids.to(torch.int32), "weights": weights}


def _logp(s):
    c = s["c"]
    T, V, n = c["T"], c["V"], c["n"]
    if own:
        import quantized_moe_expert_rl_gb300 as rl
        rl.rl_logprobs(s["x"], T, V, s["targets"], s["logprob"], s["entropy"], n, s["top_ids"], s["top_logprob"],
                       s["scratch"], s["scratch"].numel())
        return {k: s[k] for k in ("logprob", "entropy", "top_ids", "top_logprob")}
    x = s["x"].float()
    x = x - x.amax(1, keepdim=True)
    e = x.exp()
    z = e.sum(1, keepdim=True)
    logz = z.log()
    out = {"logprob": (x.gather(1, s["targets"].long()[:, None]) - logz)[:, 0],
           "entropy": (logz - (e * x).sum(1, keepdim=True) / z)[:, 0], "top_ids": None, "top_logprob": None}
    if n:
        top, ids = torch.sort(x, dim=1, descending=True, stable=True)
        out["top_ids"], out["top_logprob"] = ids[:, :n].to(torch.int32), top[:, :n] - logz
    return out


# ---- the definitions in 64 bits -----------------------------------------------------------
def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "norm":
        H, G = c["H"], c["group"]
        x = s["x"] if s["res"] is None else torch.add(s["x"].double(), s["res"].double()).to(DT[c["dtype"]])
        v = x.double()
        v = v / (torch.linalg.vector_norm(v, dim=1, keepdim=True) ** 2 / H + EPS).sqrt()
        if s["gain"] is not None:
            v = torch.einsum("th,h->th", v, s["gain"].double())
        scale = torch.stack([p.abs().max(1).values for p in v.split(G, 1)], 1) / F8_MAX
        q = v / scale.repeat_interleave(G, 1).clamp_min(1e-300)
        return {"x_out": None if s["res"] is None else x.double(), "xn": v, "q": q.float().to(F8).double(),
                "scale": scale}
    if c["op"] == "q4":
        N, K, G = c["N"], c["K"], c["group"]
        x = s["x"].float().double()
        if s["xs"] is not None:
            x = x * s["xs"].double().repeat_interleave(G, 1)
        even, odd = x[:, 0::2], x[:, 1::2]
        y = []
        for n0 in range(0, N, 16384):
            w, ws = s["w"][n0:n0 + 16384].int(), s["ws"][n0:n0 + 16384].double().repeat_interleave(G // 2, 1)
            y.append(even @ ((w % 16 - 8) * ws).t() + odd @ ((w // 16 - 8) * ws).t())
        return torch.cat(y, 1)
    if c["op"] == "moe":
        T, H, K, I = c["T"], c["H"], c["K"], c["I"]
        x = s["x"].double()
        if c["norm"]:
            x = x / (x.pow(2).sum(1, keepdim=True) / H + EPS).sqrt()
        logits = torch.einsum("th,eh->te", x, s["router"].double())
        grid, signs = s["codebook"].double(), torch.tensor(
            [[1.0 - 2.0 * (m >> j & 1) for j in range(8)] for m in range(256)], dtype=torch.float64, device="cuda")
        top = logits.topk(K, 1)
        weights = torch.exp(top.values - torch.logsumexp(top.values, 1, keepdim=True))
        y, part = torch.zeros(T, H, dtype=torch.float64, device="cuda"), H * I
        for e in sorted(set(top.indices.flatten().tolist())):
            raw = s["pool"][e].view(-1, BLOCK_BYTES)
            d = raw[:, :2].int()
            d = torch.from_numpy((d[:, 0] + 256 * d[:, 1]).cpu().numpy().astype(np.uint16).view(np.float16)
                                 .astype(np.float64)).cuda()
            w = (grid[raw[:, 2::2].int()] * signs[raw[:, 3::2].int()]).view(-1, BLOCK) * d[:, None]
            w = w.view(-1)
            t, k = (top.indices == e).nonzero(as_tuple=True)
            a, b = x[t] @ w[:part].view(I, H).t(), x[t] @ w[part:2 * part].view(I, H).t()
            y.index_add_(0, t, weights[t, k][:, None] * ((a / (1 + torch.exp(-a)) * b) @ w[2 * part:].view(H, I).t()))
        return {"y": y, "ids": None, "weights": weights}
    x = s["x"].double()
    lp = torch.log_softmax(x, 1)
    n = c["n"]
    return {"logprob": lp[torch.arange(c["T"], device="cuda"), s["targets"].long()],
            "entropy": -torch.xlogy(lp.exp(), lp.exp()).sum(1), "top_ids": None,
            "top_logprob": lp.topk(n, 1).values if n else None}
