"""Timing cases of the gate and of the dense projections around the experts.

Two operators of one MoE layer's surroundings:

* gate: router logits -> the k experts of each token and their weights (softmax or sigmoid
  scores, an additive bias that steers the choice only, groups of experts, renormalised and
  scaled weights);
* linear: y = act(x w^T + bias) + residual, the bf16 / fp16 projections beside the experts
  (attention output with its residual, router logits in fp32, a dense SwiGLU block, the
  vocabulary head).

Where ``own`` is false the operators run in plain torch in 32 bits, else through this
repository's package.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
F32_MAX = 3.4028234663852886e38


def _gate(name, T, E, k, **kw):
    c = {"name": name, "op": "gate", "T": T, "E": E, "k": k, "type": "f32", "score": "softmax", "bias": False,
         "groups": 1, "group_topk": 1, "group_score": "top2", "renormalise": True, "scale": 1.0, "masked": 0.0, "pad": 0}
    c.update(kw)
    return c


def _linear(name, T, N, K, **kw):
    c = {"name": name, "op": "linear", "T": T, "N": N, "K": K, "type": "bf16", "out": "bf16", "act": "none",
         "bias": False, "residual": False, "pad": 0}
    c.update(kw)
    return c


def listed():
    return [
        # one decode step's choice among grouped experts with a balance bias: pure latency
        _gate("gate_decode", 1, 256, 8, score="sigmoid", bias=True, groups=8, group_topk=4, scale=2.5),
        # a 512-token prefill chunk, softmax over 256 experts, as the framework's own router scores them
        _gate("gate_chunk_512", 512, 256, 8),
        # a ragged batch with few experts, a padded logits buffer, experts switched off per token (some tokens lose all)
        _gate("gate_ragged_masked", 1021, 60, 6, type="f16", renormalise=False, masked=0.15, pad=4),
        # a long chunk over many experts in bf16, where exact ties are common
        _gate("gate_many_experts", 4096, 512, 10, type="bf16", bias=True),
        # the longest chunk the framework takes, grouped sigmoid gate with a balance bias
        _gate("gate_chunk_65536", 65536, 256, 8, score="sigmoid", bias=True, groups=8, group_topk=4, scale=2.5),
        # one decode step's square projection with its residual: latency and 8 MB of weights
        _linear("linear_decode", 1, 2048, 2048, residual=True),
        # a vocabulary head for 16 sequences, logits in fp32: weight streaming
        _linear("linear_head_16", 16, 131072, 2048, out="f32"),
        # fp32 router logits of a 4096-token chunk
        _linear("linear_router_4096", 4096, 256, 2048, out="f32", bias=True),
        # odd everything: rows that start at no 16-byte boundary
        _linear("linear_odd", 333, 777, 1001, type="f16", out="f16", act="gelu", bias=True, residual=True),
        # gate and up projection of a dense SwiGLU block on a 512-token chunk
        _linear("linear_swiglu_512", 512, 4096, 2048, act="swiglu"),
        # attention output (16 heads of 256) of a 4096-token chunk, added to the residual stream
        _linear("linear_out_4096", 4096, 2048, 4096, residual=True),
        # the widest dense projection over 16384 tokens
        _linear("linear_wide_16384", 16384, 8192, 2048, act="silu", bias=True),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    if rng.random() < 0.45:
        groups = rng.choice([1, 1, 2, 4, 8, 16])
        per = _spread(rng, max(4, 8 // groups), 1024 // groups)
        E = groups * per
        T = _spread(rng, 1, min(65536, 65536 * 256 // E))
        keep = rng.randint(1, groups)
        k = rng.randint(1, min(32, keep * per))
        c = _gate("", T, E, k, type=rng.choice(["f32", "f32", "bf16", "f16"]), score=rng.choice(["softmax", "sigmoid"]),
                  bias=rng.random() < 0.5, groups=groups, group_topk=keep, group_score=rng.choice(["top2", "max"]),
                  renormalise=rng.random() < 0.7, scale=rng.choice([1.0, 2.5]),
                  masked=rng.choice([0.0, 0.0, 0.1]), pad=rng.choice([0, 0, 1, 8]))
    else:
        K = _spread(rng, 32, 8192)
        N = _spread(rng, 16, min(131072, 131072 * 2048 // K))
        T = _spread(rng, 1, 16384)
        out = rng.choice(["same", "same", "same", "f32"])
        residual = rng.random() < 0.4
        written = (2 if out == "f32" else 1) * (2 if residual else 1)
        T = max(1, min(T, 16384 * 8192 // (N * written), (16384 * 8192 * 2048) // (N * K)))
        if rng.random() < 0.6:   # most models' widths are multiples of 64; the rest stay as drawn, odd ones among them
            K, N = max(64, K // 64 * 64), max(16, N // 64 * 64)
        t = rng.choice(["bf16", "bf16", "f16"])
        act = rng.choice(["none", "none", "relu", "silu", "gelu", "gelu_tanh", "swiglu"])
        if act == "swiglu":      # two weight rows per output
            N = max(16, N // 2)
        c = _linear("", T, N, K, type=t, out=t if out == "same" else "f32", act=act, bias=rng.random() < 0.5,
                    residual=residual, pad=rng.choice([0, 0, 0, 8, 3]))
    del c["name"]
    for key in ("T", "N", "K"):   # a size that no configuration here has
        if c.get(key) == 3072:
            c[key] -= 1
    return c


# ---------------------------------------------------------------------------------------------
# inputs


def _clear_choice(c, logits, bias):
    """True for the tokens whose choice does not hang on the last bits of a 32-bit score.

    Two right implementations may round scores differently, and then rank two scores that are
    within rounding of each other differently; exact ties are kept (they go to the lower index).
    """
    l = torch.nan_to_num(logits.double(), nan=-math.inf, posinf=F32_MAX, neginf=-math.inf)
    if c["score"] == "sigmoid":
        s = torch.sigmoid(l)
    else:
        s = torch.nan_to_num(torch.softmax(l, 1), nan=0.0)
    v = s if bias is None else s + bias.double()
    size = s if bias is None else s + bias.double().abs()      # what a rounding error is relative to
    ok = torch.ones(l.shape[0], dtype=torch.bool, device=l.device)
    G = c["groups"]
    if G > 1:
        per = c["E"] // G
        top = v.view(-1, G, per).topk(min(per, 2 if c["group_score"] == "top2" else 1), 2).values.sum(2)
        rank = torch.sort(top, dim=1, descending=True, stable=True)
        if c["group_topk"] < G:
            a, b = rank.values[:, c["group_topk"] - 1], rank.values[:, c["group_topk"]]
            near = 1e-5 * size.amax(1)
            ok &= (a == b) | (a - b > near)
        keep = torch.zeros_like(top, dtype=torch.bool).scatter_(1, rank.indices[:, :c["group_topk"]], True)
        v = v.masked_fill(~keep.repeat_interleave(per, 1), -math.inf)
    n = min(c["E"], c["k"] + 1)
    best = v.topk(n, 1)
    m = size.gather(1, best.indices)
    a, b = best.values[:, :-1], best.values[:, 1:]
    return ok & ((a == b) | (a - b > 4e-6 * (m[:, :-1] + m[:, 1:]))).all(1)


def _draw_logits(c, n, popular, g):
    l = 1.5 * torch.randn(n, c["E"], device="cuda", generator=g) + popular
    l = l.to(DTYPES[c["type"]])
    if c["masked"]:
        off = torch.rand(n, c["E"], device="cuda", generator=g) < c["masked"]
        share = torch.rand(n, 1, device="cuda", generator=g)
        off |= share < 0.02                                             # tokens with nothing left
        off |= (share > 0.95) & (torch.arange(c["E"], device="cuda") >= max(1, c["k"] // 2))   # fewer than k left
        l.masked_fill_(off, -math.inf)
    return l


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *shape: torch.randn(*shape, device="cuda", generator=g)  # noqa: E731
    st = {"c": c}
    if c["op"] == "gate":
        T, E = c["T"], c["E"]
        popular = 0.5 * rand(E)                                        # experts differ in popularity
        st["bias"] = 0.1 * rand(E) if c["bias"] else None              # and the bias evens the load out
        buf = torch.zeros(T, E + c["pad"], device="cuda", dtype=DTYPES[c["type"]])
        logits = buf[:, :E]
        logits.copy_(_draw_logits(c, T, popular, g))
        for _ in range(30):
            again = (~_clear_choice(c, logits, st["bias"])).nonzero().flatten()
            if again.numel() == 0:
                break
            logits[again] = _draw_logits(c, again.numel(), popular, g)
        st["logits"] = logits
        if own:
            import quantized_grouped_gemm_gb300 as moe
            st["cfg"] = moe.gate_config(T, E, c["k"], score=c["score"], dtype=logits.dtype, groups=c["groups"],
                                        group_topk=c["group_topk"], group_score=c["group_score"],
                                        renormalise=c["renormalise"], scale=c["scale"], logits_stride=E + c["pad"])
        st["idx"] = torch.empty(T, c["k"], dtype=torch.int32, device="cuda")
        st["w"] = torch.empty(T, c["k"], dtype=torch.float32, device="cuda")
        return st
    T, N, K, t, o = c["T"], c["N"], c["K"], DTYPES[c["type"]], DTYPES[c["out"]]
    rows = 2 * N if c["act"] == "swiglu" else N
    pad = c["pad"]
    st["x"] = rand(T, K + pad).to(t)[:, :K]
    st["w"] = torch.empty(rows, K + pad, device="cuda", dtype=t).normal_(0.0, K ** -0.5, generator=g)[:, :K]
    st["bias"] = 0.5 * rand(rows) if c["bias"] else None
    st["residual"] = rand(T, N + pad).to(o)[:, :N] if c["residual"] else None
    st["y"] = torch.empty(T, N, dtype=o, device="cuda")
    if own:
        import quantized_grouped_gemm_gb300 as moe
        st["cfg"] = moe.linear_config(T, N, K, dtype=t, out_dtype=o, activation=c["act"], x_stride=K + pad,
                                      w_stride=K + pad, residual_stride=N + pad, y_stride=N)
        st["ws"] = moe.linear_workspace(st["cfg"])
    return st


# ---------------------------------------------------------------------------------------------
# one pass


def _plain_gate(st):
    c, bias = st["c"], st["bias"]
    l = torch.nan_to_num(st["logits"].float(), nan=-math.inf, posinf=F32_MAX, neginf=-math.inf)
    if c["score"] == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-l))
    else:
        m = l.amax(1, keepdim=True)
        e = torch.exp(l - torch.where(m == -math.inf, 0.0, m))
        z = e.sum(1, keepdim=True)
        s = e / torch.where(z > 0, z, 1.0)
    v = s if bias is None else s + bias
    if c["groups"] > 1:
        per = c["E"] // c["groups"]
        top = torch.sort(v.view(-1, c["groups"], per), dim=2, descending=True).values
        top = top[:, :, 0] + top[:, :, 1] if c["group_score"] == "top2" else top[:, :, 0]
        rank = torch.sort(top, dim=1, descending=True, stable=True).indices
        keep = torch.zeros_like(top, dtype=torch.bool).scatter_(1, rank[:, :c["group_topk"]], True)
        v = torch.where(keep.repeat_interleave(per, 1), v, -math.inf)
    idx = torch.sort(v, dim=1, descending=True, stable=True).indices[:, :c["k"]]
    w = s.gather(1, idx)
    if c["renormalise"]:
        z = w.sum(1, keepdim=True)
        w = w / torch.where(z > 0, z, 1.0)
    return idx.to(torch.int32), w * c["scale"]


def _plain_act(name, z):
    if name == "relu":
        return torch.clamp(z, min=0.0)
    if name == "silu":
        return z / (1.0 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if name == "swiglu":
        n = z.shape[1] // 2
        return z[:, :n] / (1.0 + torch.exp(-z[:, :n])) * z[:, n:]
    return z


def _plain_linear(st):
    z = torch.matmul(st["x"].float(), st["w"].float().t())
    if st["bias"] is not None:
        z = z + st["bias"]
    z = _plain_act(st["c"]["act"], z)
    if st["residual"] is not None:
        z = z + st["residual"].float()
    return z.to(st["y"].dtype)


def run(state):
    st = state
    if st["c"]["op"] == "gate":
        if not own:
            idx, w = _plain_gate(st)
            return {"idx": idx, "w": w}
        import quantized_grouped_gemm_gb300 as moe
        moe.moe_gate(st["cfg"], st["logits"], st["bias"], st["idx"], st["w"])
        return {"idx": st["idx"], "w": st["w"]}
    if not own:
        return {"y": _plain_linear(st)}
    import quantized_grouped_gemm_gb300 as moe
    moe.moe_linear(st["cfg"], st["x"], st["w"], st["bias"], st["residual"], st["y"], st["ws"])
    return {"y": st["y"]}


def work(case):
    c = case
    size = lambda t: 4 if t == "f32" else 2  # noqa: E731
    if c["op"] == "gate":
        T, E, k = c["T"], c["E"], c["k"]
        # a score takes about an exponential and a few sums and comparisons an expert
        return {"bytes": T * E * size(c["type"]) + (4 * E if c["bias"] else 0) + 8 * T * k, "flops": 8 * T * E}
    T, N, K = c["T"], c["N"], c["K"]
    rows = 2 * N if c["act"] == "swiglu" else N
    b = (T * K + rows * K) * size(c["type"]) + T * N * size(c["out"]) * (2 if c["residual"] else 1)
    return {"bytes": b + (4 * rows if c["bias"] else 0), "flops": 2 * T * rows * K}


# ---------------------------------------------------------------------------------------------
# the definition in 64 bits


def _exact_gate(c, logits, bias):
    l = logits.to(torch.float64).clone()
    l[torch.isnan(l)] = -math.inf
    l[l == math.inf] = F32_MAX
    if c["score"] == "sigmoid":
        s = torch.special.expit(l)
    else:
        s = torch.exp(l - torch.logsumexp(l, 1, keepdim=True))
        s[torch.isnan(s)] = 0.0
    choice = s if bias is None else s + bias.to(torch.float64)[None, :]
    if c["groups"] > 1:
        blocks = choice.unflatten(1, (c["groups"], -1))
        value = blocks.amax(2) if c["group_score"] == "max" else torch.topk(blocks, 2, dim=2).values.sum(2)
        # a group is dropped when group_topk others are better, or as good and earlier
        earlier = torch.ones(c["groups"], c["groups"], device=l.device).tril(-1).bool()[None]
        better = (value[:, None, :] > value[:, :, None]) | ((value[:, None, :] == value[:, :, None]) & earlier)
        dropped = better.sum(2) >= c["group_topk"]
        choice = blocks.masked_fill(dropped[:, :, None], -math.inf).flatten(1)
    idx = torch.argsort(choice, dim=1, descending=True, stable=True)[:, :c["k"]]
    w = torch.take_along_dim(s, idx, 1)
    if c["renormalise"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, torch.zeros_like(w))
    return {"idx": idx.to(torch.int32), "w": c["scale"] * w}


def _exact_linear(c, st):
    w64 = st["w"].to(torch.float64)
    z = torch.einsum("tk,nk->tn", st["x"].to(torch.float64), w64)
    if c["bias"]:
        z += st["bias"].to(torch.float64)
    a = c["act"]
    if a == "relu":
        z = torch.where(z > 0, z, torch.zeros_like(z))
    elif a == "silu":
        z = z * torch.special.expit(z)
    elif a == "gelu":
        z = z * torch.special.ndtr(z)
    elif a == "gelu_tanh":
        z = z * torch.special.expit(2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3))
    elif a == "swiglu":
        gate, up = z.chunk(2, 1)
        z = gate * torch.special.expit(gate) * up
    if c["residual"]:
        z = z + st["residual"].to(torch.float64)
    return {"y": z}


def exact(case, seed):
    st = prepare(case, seed)
    c = st["c"]
    if c["op"] == "gate":
        return _exact_gate(c, st["logits"], st["bias"])
    return _exact_linear(c, st)
