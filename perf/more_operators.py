"""More operators around the routed experts: what is timed, on which inputs, and the plain form of each.

Three operators that a program calls next to the routed layers, one after the other:

  matmul  product of 8-bit activations (a scale per 128 of a row) and 8-bit weights (a scale per block
          of 128 x 128), from one row to a prompt chunk: projections, an output head
  gated   the gated half of a feed-forward block in the same format: both projections, the activation
          and their product, again in 8 bits with a scale per 128 (what the down projection reads)
  sample  the next token of each row of logits: temperature, top-k, top-p and min-p, drawn by a given
          random number

`run` computes the plain form with elementary torch operations where `own` is false, and calls the
framework where it is true.  The sizes are those of the framework's workloads (hidden 2048,
intermediate 512, chunks of up to 2048 tokens, vocabulary of 131072) and generic ones.
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
F8 = torch.float8_e4m3fn
F8_MAX = 448.0
G = 128


def listed():
    return [
        # a shared expert's down projection for one decoded token, added to the routed experts' sum: latency
        dict(name="matmul 2048x512 1 token", op="matmul", N=2048, K=512, T=1, y="f32", res=True),
        # the output head for eight sequences: the largest matrix a decode step reads
        dict(name="matmul head 8 tokens", op="matmul", N=131072, K=2048, T=8, y="f32", res=False),
        # a projection of odd height, a width that ends inside a block, a ragged number of rows
        dict(name="matmul odd 77 tokens", op="matmul", N=10007, K=1040, T=77, y="f16", res=False),
        # a wide dense projection of a long prompt: the tensor cores
        dict(name="matmul 8192x8192 4096 tokens", op="matmul", N=8192, K=8192, T=4096, y="bf16", res=False),
        # a shared expert's gate and up projections for one decoded token: latency
        dict(name="gated 512x2048 1 token", op="gated", I=512, K=2048, T=1, out="f8"),
        # the same kind of layer with ragged sizes and a 16-bit output
        dict(name="gated odd 50 tokens", op="gated", I=1016, K=784, T=50, out="bf16"),
        # a shared expert over a prompt chunk
        dict(name="gated 512x2048 2048 tokens", op="gated", I=512, K=2048, T=2048, out="f8"),
        # a dense feed-forward layer over a long prompt
        dict(name="gated 8192x4096 4096 tokens", op="gated", I=8192, K=4096, T=4096, out="f8"),
        # one sequence: the last step of a decoded token
        dict(name="sample 1 row k p", op="sample", T=1, V=131072, dtype="f32", shape="peaked", heat=0.8, k=50, p=0.9, m=0.0),
        # thirty-two sequences with settings of their own, 16-bit logits (exact ties), odd vocabulary
        dict(name="sample 32 rows mixed", op="sample", T=32, V=100003, dtype="bf16", shape="mixed", heat=0.0, k=-1, p=-1.0,
             m=-1.0),
        # a rollout of many sequences from the model's own distribution, nothing left out
        dict(name="sample 512 rows all", op="sample", T=512, V=131072, dtype="f32", shape="mixed", heat=1.0, k=0, p=1.0, m=0.0),
        # the same with a nucleus, on rows from peaked to nearly flat
        dict(name="sample 512 rows p", op="sample", T=512, V=131072, dtype="f32", shape="mixed", heat=1.0, k=0, p=0.95, m=0.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["matmul", "gated", "sample"])
    if op == "sample":
        V = _log(rng, 500, 131072)
        return dict(op=op, T=_log(rng, 1, 512), V=V, dtype=rng.choice(["f32", "f16", "bf16"]),
                    shape=rng.choice(["peaked", "broad", "mixed"]), heat=rng.choice([0.0, 0.3, 0.7, 1.0, 1.3]),
                    k=rng.choice([0, 0, -1, _log(rng, 1, V)]), p=rng.choice([1.0, -1.0, 0.3, 0.8, 0.95]),
                    m=rng.choice([0.0, 0.0, -1.0, 0.02, 0.2]))
    K = 16 * _log(rng, 2, 512)
    T = _log(rng, 1, 4096)
    rows = _log(rng, 40, 131072)
    # no more operations than the largest listed case, nor more weights or outputs than the listed ones
    rows = max(40, min(rows, int(2 ** 39 / (2 * T * K)), 2 ** 28 // K, 2 ** 27 // T))
    if op == "matmul":
        return dict(op=op, N=rows, K=K, T=T, y=rng.choice(["f32", "f16", "bf16"]), res=rng.random() < 0.4)
    out = rng.choice(["f8", "f8", "f32", "f16", "bf16"])
    return dict(op=op, I=rows // 2 // 16 * 16 or 16 if out == "f8" else rows // 2, K=K, T=T, out=out)


def work(c):
    """Bytes and operations that no form of the operator can do without."""
    if c["op"] == "sample":
        T, V = c["T"], c["V"]
        return {"bytes": T * V * DT[c["dtype"]].itemsize + T * 28, "flops": 5.0 * T * V}
    T, K = c["T"], c["K"]
    rows = c["N"] if c["op"] == "matmul" else 2 * c["I"]
    read = rows * K + T * K + 4 * (-(-K // G)) * (T + -(-rows // G))
    if c["op"] == "matmul":
        return {"bytes": read + T * rows * DT[c["y"]].itemsize * (2 if c["res"] else 1), "flops": 2.0 * T * rows * K}
    I = c["I"]
    write = T * (I + 4 * -(-I // G)) if c["out"] == "f8" else T * I * DT[c["out"]].itemsize
    return {"bytes": read + write, "flops": 2.0 * T * rows * K}


# ---- inputs -------------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 6007 + 29)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _rand(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda", dtype=torch.float32)


def _weights(g, N, K):
    """An 8-bit matrix whose blocks use the type's range, and its scales."""
    w = torch.empty(N, K, dtype=F8, device="cuda")
    for n in range(0, N, 16384):
        part = w[n:n + 16384]
        part.copy_((100 * _randn(g, *part.shape)).clamp_(-F8_MAX, F8_MAX))
    return w, (0.5 + _rand(g, -(-N // G), -(-K // G))) * (0.02 / 100)


def _groups(v):
    """Rows [T][K] as [T][groups][128], the last group filled up with zeros."""
    T, K = v.shape
    return torch.nn.functional.pad(v, (0, -K % G)).view(T, -1, G)


def prepare(c, seed):
    g, s = _gen(seed), {"c": c}
    empty = lambda *shape, dtype=torch.float32: torch.empty(*shape, dtype=dtype, device="cuda")  # noqa: E731
    T = c["T"]
    if c["op"] == "sample":
        V = c["V"]
        # next-token logits: a background and a few likely candidates, or hardly any preference
        peaked, broad = 2.0 * _randn(g, T, V) - 4, 1.0 * _randn(g, T, V)
        peaked.scatter_(1, torch.randint(0, V, (T, 12), generator=g, device="cuda"), 9 + 3 * _randn(g, T, 12))
        if c["shape"] == "mixed":
            x = torch.where(_rand(g, T, 1) < 0.75, peaked, broad)
        else:
            x = peaked if c["shape"] == "peaked" else broad
        s["x"] = x.to(DT[c["dtype"]])
        s["u"] = _rand(g, T)
        pick = lambda *v: torch.tensor(v, device="cuda")[torch.randint(0, len(v), (T,), generator=g, device="cuda")]  # noqa: E731
        # a setting for all rows, or (negative; temperature 0) one for each row
        s["heat"] = pick(0.0, 0.3, 0.7, 1.0, 1.2) if c["heat"] == 0 else torch.full((T,), c["heat"], device="cuda")
        s["k"] = pick(0, 1, 20, 50, 200).int() if c["k"] < 0 else \
            torch.full((T,), c["k"], dtype=torch.int32, device="cuda") if c["k"] else None
        s["p"] = pick(1.0, 0.5, 0.9, 0.95) if c["p"] < 0 else torch.full((T,), c["p"], device="cuda") if c["p"] < 1 else None
        s["m"] = pick(0.0, 0.05, 0.1) if c["m"] < 0 else torch.full((T,), c["m"], device="cuda") if c["m"] else None
        s["ids"], s["logprob"] = empty(T, dtype=torch.int32), empty(T)
        return s
    K = c["K"]
    x = _randn(g, T, K) * (1 + 15 * (_rand(g, K) < 0.01))
    s["xs"] = _groups(x).abs().amax(2).clamp_min(1e-20) / F8_MAX
    s["x"] = (_groups(x) / s["xs"][:, :, None]).clamp(-F8_MAX, F8_MAX).view(T, -1)[:, :K].to(F8).contiguous()
    if c["op"] == "matmul":
        N = c["N"]
        s["w"], s["ws"] = _weights(g, N, K)
        s["res"] = _randn(g, T, N).to(DT[c["y"]]) if c["res"] else None
        s["y"] = empty(T, N, dtype=DT[c["y"]])
    else:
        I = c["I"]
        s["wg"], s["sg"] = _weights(g, I, K)
        s["wu"], s["su"] = _weights(g, I, K)
        s["h"] = empty(T, I, dtype=DT[c["out"]]) if c["out"] != "f8" else None
        s["q"] = empty(T, I, dtype=F8) if c["out"] == "f8" else None
        s["scale"] = empty(T, -(-I // G)) if c["out"] == "f8" else None
    return s


# ---- the operators ------------------------------------------------------------------------
def run(s):
    return {"matmul": _matmul, "gated": _gated, "sample": _sample}[s["c"]["op"]](s)


def _rows(x, xs):
    return (_groups(x.float()) * xs[:, :, None]).view(x.shape[0], -1)[:, :x.shape[1]]


def _matrix(w, ws):
    N, K = w.shape
    return w.float() * ws.repeat_interleave(G, 0)[:N].repeat_interleave(G, 1)[:, :K]


def _matmul(s):
    c = s["c"]
    if own:
        import quantized_moe_expert_rl_gb300 as rl
        rl.rl_f8_matmul(s["w"], s["ws"], s["x"], s["xs"], s["y"], c["T"], c["N"], c["K"], res=s["res"])
        return s["y"]
    y = _rows(s["x"], s["xs"]) @ _matrix(s["w"], s["ws"]).t()
    if s["res"] is not None:
        y = y + s["res"].float()
    return y.to(DT[c["y"]])


def _gated(s):
    c = s["c"]
    if own:
        import quantized_moe_expert_rl_gb300 as rl
        rl.rl_f8_gated(s["wg"], s["sg"], s["wu"], s["su"], s["x"], s["xs"], c["T"], c["I"], c["K"], h=s["h"], q=s["q"],
                       scale=s["scale"])
        return {k: s[k] for k in ("h", "q", "scale")}
    x = _rows(s["x"], s["xs"])
    a, b = x @ _matrix(s["wg"], s["sg"]).t(), x @ _matrix(s["wu"], s["su"]).t()
    h = a * torch.sigmoid(a) * b
    if c["out"] != "f8":
        return {"h": h.to(DT[c["out"]]), "q": None, "scale": None}
    v = _groups(h)
    scale = v.abs().amax(2) / F8_MAX
    q = torch.where(scale[:, :, None] > 0, v / scale[:, :, None], torch.zeros_like(v)).clamp(-F8_MAX, F8_MAX)
    return {"h": None, "q": q.view(c["T"], -1)[:, :c["I"]].to(F8), "scale": scale}


def _sample(s):
    """The tokens in descending order (equal logits: the lower index first); the first k; of those the
    shortest run that holds a share p of the probability; of those the ones at least m times as probable
    as the first.  Then the first token in the vocabulary's order at which the sum of the kept ones'
    probabilities passes u.  In 64 bits: a token next to a border is in or out."""
    if own:
        import quantized_moe_expert_rl_gb300 as rl
        c = s["c"]
        rl.rl_sample(s["x"], c["T"], c["V"], s["u"], s["ids"], temperature=s["heat"], top_k=s["k"], top_p=s["p"],
                     min_p=s["m"], logprob=s["logprob"])
        return {"ids": s["ids"], "logprob": s["logprob"]}
    T, V = s["x"].shape
    top, order = torch.sort(s["x"], dim=1, descending=True, stable=True)
    heat = s["heat"].double()[:, None]
    z = (top.double() - top[:, :1].double()) / torch.where(heat > 0, heat, torch.ones_like(heat))
    at = torch.arange(V, device=z.device)[None, :]
    kept = (at < 1) | (heat > 0)
    if s["k"] is not None:
        k = s["k"][:, None]
        kept = kept & ((at < k) | (k <= 0))
    e = torch.where(kept, z.exp(), torch.zeros_like(z))
    if s["p"] is not None:
        before = e.cumsum(1) - e
        kept = kept & ((at < 1) | (before < s["p"].double()[:, None] * e.sum(1, keepdim=True)) | (s["p"][:, None] >= 1))
        del before
    if s["m"] is not None:
        kept = kept & ((at < 1) | (z >= s["m"].double()[:, None].log()))
    e = torch.where(kept, e, torch.zeros_like(e))
    mass = torch.zeros_like(e).scatter_(1, order, e)
    total = e.sum(1, keepdim=True)
    upto = mass.cumsum(1)
    # the first place where the running sum passes u; where rounding left none, the last kept token
    ids = torch.minimum((upto <= s["u"].double()[:, None] * total).sum(1), (at * (mass > 0)).amax(1))
    logprob = mass.gather(1, ids[:, None]).log() - total.log()
    return {"ids": ids.to(torch.int32), "logprob": logprob[:, 0].float()}


# ---- the definitions in 64 bits -----------------------------------------------------------
def _product(x, xs, w, ws):
    """Block by block of the shared dimension, the scales on the block's sums."""
    T, N = x.shape[0], w.shape[0]
    y = torch.zeros(T, N, dtype=torch.float64, device="cuda")
    for n in range(0, N, 8192):
        part = w[n:n + 8192]
        rows = torch.arange(n, n + part.shape[0], device="cuda") // G
        for b in range(xs.shape[1]):
            d = x[:, G * b:G * b + G].float().double() @ part[:, G * b:G * b + G].float().double().t()
            y[:, n:n + 8192] += d * xs[:, b, None].double() * ws[rows, b].double()
    return y


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "matmul":
        y = _product(s["x"], s["xs"], s["w"], s["ws"])
        return y if s["res"] is None else torch.add(y, s["res"].double())
    if c["op"] == "gated":
        a = _product(s["x"], s["xs"], s["wg"], s["sg"])
        h = a / (1 + torch.exp(-a)) * _product(s["x"], s["xs"], s["wu"], s["su"])
        if c["out"] != "f8":
            return {"h": h, "q": None, "scale": None}
        scale = torch.stack([v.abs().max(1).values for v in h.split(G, 1)], 1) / F8_MAX
        q = h / scale.repeat_interleave(G, 1)[:, :c["I"]].clamp_min(1e-300)
        return {"h": None, "q": q.float().to(F8).double(), "scale": scale}
    ids, logprob = [], []
    for t in range(c["T"]):
        x, heat = s["x"][t].double(), float(s["heat"][t])
        if heat <= 0:
            ids.append(int((x == x.max()).nonzero()[0, 0]))
            logprob.append(0.0)
            continue
        order = torch.argsort(-x, stable=True)
        n = c["V"]
        if s["k"] is not None and 0 < int(s["k"][t]) < n:
            n = int(s["k"][t])
        lp = torch.log_softmax(x[order[:n]] / heat, 0)
        if s["p"] is not None and float(s["p"][t]) < 1:
            # what is left behind a token, summed from the least probable one up
            behind = lp.exp().flip(0).cumsum(0).flip(0)
            n = max(1, int((behind > (1 - s["p"][t].double()) * behind[0]).sum()))
        if s["m"] is not None and float(s["m"][t]) > 0:
            n = min(n, max(1, int((lp - lp[0] >= math.log(float(s["m"][t]))).sum())))
        chosen, _ = order[:n].sort()
        p = torch.softmax(x[chosen] / heat, 0)
        at = min(int(torch.searchsorted(p.cumsum(0), s["u"][t].double().view(1), right=True)), n - 1)
        ids.append(int(chosen[at]))
        logprob.append(math.log(float(p[at])))
    return {"ids": torch.tensor(ids, dtype=torch.int32), "logprob": torch.tensor(logprob, dtype=torch.float64)}
