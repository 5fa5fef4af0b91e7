"""More layer steps, as cases that can be timed and compared: what a delta-rule
model needs around its mixers to be trained from tokens and to be decoded.

Four operators, each in its directions and types: the gated delta rule token
by token over a pool of state slots, the causal conv1d's tokens over a pool of
window slots, layer norm (forward with residual, 16 / 32-bit and e4m3 outputs;
backward) and the embedding lookup with its gradient.  ``run`` computes a case
with elementary torch operations (``own`` false) or through
``context_merge_gb300.cpdr.Context`` (``own`` true); ``exact`` computes it in
64 bits from the definition.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-5
E4M3_MAX = 448.0
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # decoding one sequence at 16 heads x 128: latency counts
        dict(name="delta_n1_h16_d128", op="delta", dtype="bf16", gate="gdn", seqs=1, longest=1, mixed=False, empty=0,
             slots=4, H=16, G=1, d=128, v_first=False),
        # decoding a batch of 64 rows, 3 of them empty, with the per-dim gate and 32 heads
        dict(name="delta_kda_n64_h32_d128", op="delta", dtype="bf16", gate="kda", seqs=61, longest=1, mixed=True,
             empty=3, slots=96, H=32, G=1, d=128, v_first=False),
        # checking 1 to 8 drafted tokens for each of 48 sequences, 32 query heads on 16 states, [dv, dk] states
        dict(name="delta_drafted_s48_l8_h16_hq32", op="delta", dtype="bf16", gate="gdn", seqs=48, longest=8,
             mixed=False, empty=5, slots=64, H=16, G=2, d=128, v_first=True),
        # the largest batch: 512 sequences
        dict(name="delta_n512_h16_d128", op="delta", dtype="bf16", gate="gdn", seqs=512, longest=1, mixed=True,
             empty=0, slots=640, H=16, G=1, d=128, v_first=False),
        # the convolution of the q, k, v projections (3 x 16 heads x 128) before them: a small batch
        dict(name="conv_n8_c6144_w4", op="conv", dtype="bf16", seqs=8, longest=1, mixed=False, empty=0, slots=16,
             channels=6144, W=4, act="silu", bias=False),
        # and a large one, with 12 empty rows
        dict(name="conv_n512_c6144_w4", op="conv", dtype="bf16", seqs=500, longest=1, mixed=True, empty=12, slots=640,
             channels=6144, W=4, act="silu", bias=True),
        # decoding a batch of 8: the norm before a projection, one launch, latency counts
        dict(name="layernorm_r8_w2048", op="norm", dtype="bf16", rows=8, width=2048, residual=True, bias=True,
             e4m3=False),
        # prefill of 32768 tokens at 32 heads x 128: the norm whose 8-bit output an e4m3 projection reads
        dict(name="layernorm_e4m3_r32768_w4096", op="norm", dtype="bf16", rows=32768, width=4096, residual=True,
             bias=True, e4m3=True),
        # training: the norm's gradients, an odd number of rows, with the residual stream's gradient added
        dict(name="layernorm_bwd_r49151_w2048", op="norm_bwd", dtype="bf16", rows=49151, width=2048, bias=True,
             dsum=True),
        # training: the embedding of a batch of 262144 tokens, scaled by the root of the width
        dict(name="embed_n262144_v131072_w2048", op="embed", dtype="bf16", n=262144, vocab=131072, width=2048,
             scale=math.sqrt(2048.0), zipf=True, pad=0),
        # fine-tuning: the gradient for a short packed batch with padding, an odd vocabulary, an fp32 table
        dict(name="embed_bwd_fp32_n1000_v32003_w1360", op="embed_bwd", dtype="fp32", n=1000, vocab=32003, width=1360,
             scale=1.0, zipf=True, pad=24),
        # training: the gradient of a batch of 131072 tokens, the most frequent one in every twelfth place
        dict(name="embed_bwd_n131072_v131072_w2048", op="embed_bwd", dtype="bf16", n=131072, vocab=131072, width=2048,
             scale=1.0, zipf=True, pad=0),
    ]


def _log(rng, lo, hi, mult=1):
    x = math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999 * mult)))
    return max(lo, min(hi, int(x) // mult * mult))


def draw(rng):
    op = rng.choice(["delta", "delta", "delta", "conv", "norm", "norm", "norm_bwd", "embed", "embed_bwd", "embed_bwd"])
    if op in ("delta", "conv"):
        c = dict(op=op, dtype=rng.choice(["bf16", "bf16", "fp32"]), seqs=_log(rng, 1, 512),
                 longest=rng.choice([1, 1, _log(rng, 1, 128)]), mixed=rng.random() < 0.5)
        if op == "delta":
            H, d = _log(rng, 1, 32), rng.choice([128, 128, 64])
            c.update(gate=rng.choice(["gdn", "kda"]), H=H, d=d, G=rng.choice([1, 1, 2, 3, 4]), v_first=rng.random() < 0.5)
            most = min(4096, (1 << 27) // (H * d * d))   # tokens whose states are the largest listed case's
        else:
            c.update(channels=_log(rng, 64, 8192, 8), W=rng.choice([2, 3, 4, 4, 4, 8]), act=rng.choice(["silu", "none"]),
                     bias=rng.random() < 0.5)
            most = min(4096, (1 << 21) // c["channels"])
        while sum(_counts(c)) > most:
            if c["longest"] > 1 and c["longest"] >= c["seqs"]:
                c["longest"] = max(1, c["longest"] // 2)
            else:
                c["seqs"] = max(1, c["seqs"] * 2 // 3)
        c.update(empty=rng.randrange(0, max(1, c["seqs"] // 4) + 1), slots=c["seqs"] + rng.randrange(1, 129))
        return c
    if op in ("norm", "norm_bwd"):
        width = rng.choice([_log(rng, 8, 8192, 8), _log(rng, 1024, 16384, 8)])
        rows = _log(rng, 1, max(2, (1 << 26) // width))
        c = dict(op=op, rows=rows, width=width, bias=rng.random() < 0.7)
        if op == "norm_bwd":
            return dict(c, dtype=rng.choice(["bf16", "bf16", "fp32"]), dsum=rng.random() < 0.5)
        e4m3 = rng.random() < 0.4
        return dict(c, dtype="bf16" if e4m3 else rng.choice(["bf16", "fp32"]), residual=rng.random() < 0.6, e4m3=e4m3)
    width = _log(rng, 64, 8192, 8)
    most = 1 << 27
    n = _log(rng, 1, min(262144, most // width))
    return dict(op=op, dtype=rng.choice(["bf16", "bf16", "fp32"]), n=n, vocab=_log(rng, 1000, min(262144, most // width)),
                width=width, scale=rng.choice([1.0, math.sqrt(width)]), zipf=rng.random() < 0.7,
                pad=rng.randrange(0, n // 8 + 1))


def _counts(case):
    """Tokens of each sequence: 1 to `longest`, a fixed function of the case."""
    return [1 + (7 * i * i + 3 * i + 5) % case["longest"] for i in range(case["seqs"])]


# ------------------------------------------------------------------ inputs
def _zipf(vocab):
    """Frequencies of the tokens of a text, 1 / (rank + 2.7), in 64 bits on the CPU."""
    p = 1.0 / (torch.arange(vocab, dtype=torch.float64) + 2.7)
    return p / p.sum()


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device=DEV)

    def perm(n):
        return torch.randperm(n, generator=gen, device=DEV)

    op, dt = case["op"], DTYPES[case["dtype"]]
    s = {"case": case}
    if op in ("delta", "conv"):
        # which slot each row continues: sequence after sequence or in mixed order, empty rows among them or behind
        chosen, counts = perm(case["slots"])[:case["seqs"]], torch.tensor(_counts(case), device=DEV)
        slots = torch.cat([chosen.repeat_interleave(counts), torch.full((case["empty"],), -1, device=DEV)])
        if case["mixed"]:
            slots = slots[perm(slots.numel())]
        s["slots"] = slots.to(torch.int32)
        # the rows of every turn: each sequence's first token, each one's second, ...
        order = torch.argsort(slots, stable=True)
        at = torch.arange(slots.numel(), device=DEV)
        first = torch.searchsorted(slots[order], slots[order])
        turn = torch.empty_like(at)
        turn[order] = at - first
        s["turns"] = [torch.nonzero((turn == j) & (slots >= 0))[:, 0] for j in range(max(_counts(case)))]
        n = slots.numel()
        if op == "delta":
            H, G, d = case["H"], case["G"], case["d"]
            for name, heads in (("q", H * G), ("k", H)):
                t = randn(n, heads, d)
                s[name] = (t / t.norm(dim=-1, keepdim=True)).to(dt)
            s["v"] = randn(n, H, d).to(dt)
            s["beta"] = torch.sigmoid(randn(n, H)).to(dt)
            if case["gate"] == "gdn":
                s["g"] = torch.nn.functional.logsigmoid(4.0 + 0.5 * randn(n, H))
            else:
                s["g"] = torch.nn.functional.logsigmoid(3.0 + randn(n, H, d))
            s["state"] = 0.3 * randn(case["slots"], H, d, d)
            s["o"] = torch.zeros(n, H * G, d, device=DEV, dtype=dt)
        else:
            C, W = case["channels"], case["W"]
            s["x"] = randn(n, C).to(dt)
            s["w"] = randn(C, W) / math.sqrt(W)
            s["b"] = 0.1 * randn(C) if case["bias"] else None
            s["state"] = randn(case["slots"], W - 1, C).to(dt)
            s["y"] = torch.zeros(n, C, device=DEV, dtype=dt)
        s["state_out"] = s["state"].clone()
    elif op in ("norm", "norm_bwd"):
        rows, width = case["rows"], case["width"]
        x = randn(rows, width)
        x *= torch.exp(0.5 * randn(rows, 1))       # rows of differing size and mean, as a residual stream has
        x += 0.5 * randn(rows, 1)
        s["x"] = x.to(dt)
        s["w"] = 1.0 + 0.2 * randn(width)
        s["b"] = 0.1 * randn(width) if case["bias"] else None
        if op == "norm":
            s["r"] = randn(rows, width).to(dt) if case["residual"] else None
        else:
            s["dy"] = randn(rows, width).to(dt)
            s["dsum"] = randn(rows, width).to(dt) if case["dsum"] else None
    else:
        n, V, D = case["n"], case["vocab"], case["width"]
        u = torch.rand(n, generator=gen, device=DEV, dtype=torch.float64)
        tokens = torch.searchsorted(_zipf(V).cumsum(0).to(DEV), u) if case["zipf"] else (u * V).long()
        tokens = tokens.clamp(max=V - 1).to(torch.int32)
        if case["pad"]:
            tokens[n - case["pad"]:] = -1          # padding behind the last sequence
        s["tokens"] = tokens
        s["live"] = torch.nonzero(tokens >= 0)[:, 0]
        if op == "embed":
            s["table"] = (0.02 * randn(V, D)).to(dt)
        else:
            s["dy"] = randn(n, D).to(dt)
    if own:
        _prepare_own(s)
    return s


def _prepare_own(s):
    """The context, workspaces and output buffers that a user's program keeps between calls."""
    from context_merge_gb300 import cpdr

    case, op = s["case"], s["case"]["op"]
    f32 = torch.float32
    if op == "delta":
        s["ctx"] = cpdr.Context(1, 1, case["H"], case["d"], 1, gate=case["gate"], dtype=case["dtype"],
                                scale=case["d"] ** -0.5, Hq=case["H"] * case["G"], state_v_first=case["v_first"])
        return
    ctx = s["ctx"] = cpdr.Context(1, 1, 1, 64, 1, dtype=case["dtype"], conv_width=case.get("W", 0))
    if op == "norm":
        x = s["x"]
        s["s"] = torch.empty_like(x) if case["residual"] else None
        s["y"] = None if case["e4m3"] else torch.empty_like(x)
        s["y8"] = torch.empty(x.shape, device=DEV, dtype=torch.float8_e4m3fn) if case["e4m3"] else None
        s["ys"] = torch.empty(x.shape[0], device=DEV, dtype=f32) if case["e4m3"] else None
    elif op == "norm_bwd":
        s["out"] = dict(ds=torch.empty_like(s["x"]), dweight=torch.empty_like(s["w"]),
                        **({"dbias": torch.empty_like(s["w"])} if case["bias"] else {}))
        s["ws"] = torch.empty(ctx.layernorm_bwd_workspace_bytes(case["rows"], case["width"]), device=DEV,
                              dtype=torch.uint8)
    elif op == "embed":
        s["y"] = torch.empty(case["n"], case["width"], device=DEV, dtype=DTYPES[case["dtype"]])
    elif op == "embed_bwd":
        s["dtable"] = torch.empty(case["vocab"], case["width"], device=DEV, dtype=DTYPES[case["dtype"]])
        s["ws"] = torch.empty(ctx.embed_bwd_workspace_bytes(case["n"], case["vocab"], case["width"]), device=DEV,
                              dtype=torch.uint8)


# ------------------------------------------------------------------ one pass
def run(state):
    op = state["case"]["op"]
    return (_OWN if own else _PLAIN)[op](state)


def _own_delta(s):
    s["ctx"].delta_step(s["q"], s["k"], s["v"], s["beta"], s["g"], s["state"], s["o"], slots=s["slots"],
                        state_out=s["state_out"])
    return {"o": s["o"], "state": s["state_out"]}


def _own_conv(s):
    s["ctx"].conv1d_step(s["x"], s["w"], s["b"], s["state"], s["y"], slots=s["slots"], state_out=s["state_out"],
                         activation=s["case"]["act"])
    return {"y": s["y"], "state": s["state_out"]}


def _own_norm(s):
    s["ctx"].layernorm_fwd(s["x"], s["w"], bias=s["b"], residual=s["r"], sum_out=s["s"], y=s["y"], y8=s["y8"],
                           scale=s["ys"], eps=EPS)
    out = {"y8": s["y8"], "scale": s["ys"]} if s["case"]["e4m3"] else {"y": s["y"]}
    if s["s"] is not None:
        out["s"] = s["s"]
    return out


def _own_norm_bwd(s):
    return s["ctx"].layernorm_bwd(s["x"], s["w"], s["dy"], dsum=s["dsum"], eps=EPS, out=s["out"], workspace=s["ws"])


def _own_embed(s):
    s["ctx"].embed_fwd(s["tokens"], s["table"], s["y"], scale=s["case"]["scale"])
    return s["y"]


def _own_embed_bwd(s):
    return s["ctx"].embed_bwd(s["tokens"], s["dy"], s["dtable"], scale=s["case"]["scale"], workspace=s["ws"])


_OWN = dict(delta=_own_delta, conv=_own_conv, norm=_own_norm, norm_bwd=_own_norm_bwd, embed=_own_embed,
            embed_bwd=_own_embed_bwd)


def _plain_delta(s):
    """Every sequence's next token at once, turn after turn."""
    case = s["case"]
    H, G, d = case["H"], case["G"], case["d"]
    state = s["state"]
    for rows in s["turns"]:
        at = s["slots"][rows].long()
        S = state[at]
        if case["v_first"]:
            S = S.transpose(2, 3)
        q, k, v = (s[name][rows].float() for name in ("q", "k", "v"))
        a = torch.exp(s["g"][rows]).reshape(len(rows), H, -1, 1)
        S = a * S
        delta = s["beta"][rows].float()[..., None] * (v - (k[..., None] * S).sum(2))
        S = S + k[..., None] * delta[:, :, None, :]
        o = (q.reshape(-1, H, G, d) @ S).reshape(-1, H * G, d) * d ** -0.5
        s["o"][rows] = o.to(s["o"].dtype)
        s["state_out"][at] = S.transpose(2, 3) if case["v_first"] else S
        state = s["state_out"]
    return {"o": s["o"], "state": s["state_out"]}


def _plain_conv(s):
    state = s["state"]
    for rows in s["turns"]:
        at = s["slots"][rows].long()
        x = torch.cat([state[at], s["x"][rows][:, None]], 1)
        z = (x.float() * s["w"].t()).sum(1)
        if s["b"] is not None:
            z = z + s["b"]
        if s["case"]["act"] == "silu":
            z = z / (1.0 + torch.exp(-z))
        s["y"][rows] = z.to(s["y"].dtype)
        s["state_out"][at] = x[:, 1:]
        state = s["state_out"]
    return {"y": s["y"], "state": s["state_out"]}


def _plain_norm(s):
    t = s["x"].float()
    out = {}
    if s["r"] is not None:
        t = t + s["r"].float()
        out["s"] = t.to(s["x"].dtype)
    t = t - t.mean(dim=1, keepdim=True)
    n = t * torch.rsqrt((t * t).mean(dim=1, keepdim=True) + EPS) * s["w"]
    if s["b"] is not None:
        n = n + s["b"]
    if s["case"]["e4m3"]:
        scale = (n.abs().amax(dim=1) / E4M3_MAX).clamp(min=2.0 ** -126)
        out["y8"] = (n / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        out["scale"] = scale
    else:
        out["y"] = n.to(s["x"].dtype)
    return out


def _plain_norm_bwd(s):
    t, dy = s["x"].float(), s["dy"].float()
    t = t - t.mean(dim=1, keepdim=True)
    rstd = torch.rsqrt((t * t).mean(dim=1, keepdim=True) + EPS)
    xh = t * rstd
    u = dy * s["w"]
    ds = rstd * (u - u.mean(dim=1, keepdim=True) - xh * (u * xh).mean(dim=1, keepdim=True))
    if s["dsum"] is not None:
        ds = ds + s["dsum"].float()
    out = {"ds": ds.to(s["x"].dtype), "dweight": (dy * xh).sum(dim=0)}
    if s["b"] is not None:
        out["dbias"] = dy.sum(dim=0)
    return out


def _plain_embed(s):
    live = s["live"]
    y = torch.zeros(s["case"]["n"], s["case"]["width"], device=DEV, dtype=s["table"].dtype)
    y[live] = (s["table"][s["tokens"][live].long()].float() * s["case"]["scale"]).to(y.dtype)
    return y


def _plain_embed_bwd(s):
    live = s["live"]
    t = torch.zeros(s["case"]["vocab"], s["case"]["width"], device=DEV)
    t.index_add_(0, s["tokens"][live], s["dy"][live].float() * s["case"]["scale"])
    return t.to(s["dy"].dtype)


_PLAIN = dict(delta=_plain_delta, conv=_plain_conv, norm=_plain_norm, norm_bwd=_plain_norm_bwd, embed=_plain_embed,
              embed_bwd=_plain_embed_bwd)


# ------------------------------------------------------------------ work
def work(case):
    op = case["op"]
    es = 4 if case["dtype"] == "fp32" else 2
    if op == "delta":
        H, G, d, live = case["H"], case["G"], case["d"], sum(_counts(case))
        return {"bytes": case["seqs"] * H * d * d * 8 + live * H * (es * (2 * G * d + 2 * d + 1) + 4 * (d if case["gate"] == "kda" else 1))
                + 4 * (live + case["empty"]), "flops": live * H * d * d * (5 + 2 * G)}
    if op == "conv":
        C, W, live = case["channels"], case["W"], sum(_counts(case))
        return {"bytes": es * C * (2 * live + 2 * (W - 1) * case["seqs"]) + 4 * C * (W + case["bias"])
                + 4 * (live + case["empty"]), "flops": live * C * (2 * W + 5)}
    if op == "norm":
        n, w = case["rows"] * case["width"], 4 * case["width"]
        return {"bytes": n * (es + (2 * es if case["residual"] else 0) + (1 if case["e4m3"] else es))
                + w * (1 + case["bias"]) + (4 * case["rows"] if case["e4m3"] else 0), "flops": 8 * n}
    if op == "norm_bwd":
        n, w = case["rows"] * case["width"], 4 * case["width"]
        return {"bytes": n * es * (4 if case["dsum"] else 3) + w * (2 + case["bias"]), "flops": 14 * n}
    n, V, D, live = case["n"], case["vocab"], case["width"], case["n"] - case["pad"]
    if op == "embed":
        # the table's rows that occur, as the tokens' distribution lets expect
        p = _zipf(V) if case["zipf"] else torch.full((V,), 1.0 / V, dtype=torch.float64)
        rows = float((1.0 - torch.exp(live * torch.log1p(-p))).sum())
        return {"bytes": es * D * (n + rows) + 4 * n, "flops": live * D}
    return {"bytes": es * D * (live + V) + 4 * n, "flops": live * D}


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    op = case["op"]
    d = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor) and v.is_floating_point()}
    if op in ("delta", "conv"):
        state = d["state"]
        out = d["o"] if op == "delta" else d["y"]
        for i, slot in enumerate(s["slots"].tolist()):
            if slot < 0:
                continue
            if op == "delta":
                out[i], state[slot] = _exact_token(case, d, i, state[slot])
                continue
            window = torch.cat([state[slot], d["x"][i:i + 1]])
            z = torch.einsum("wc,cw->c", window, d["w"]) + (d["b"] if s["b"] is not None else 0.0)
            out[i] = z * torch.sigmoid(z) if case["act"] == "silu" else z
            state[slot] = window[1:]
        return {"o" if op == "delta" else "y": out, "state": state}
    if op == "norm":
        t = d["x"] + d["r"] if s["r"] is not None else d["x"]
        var, mean = torch.var_mean(t, dim=1, unbiased=False, keepdim=True)
        n = (t - mean) / (var + EPS) ** 0.5 * d["w"] + (d["b"] if s["b"] is not None else 0.0)
        out = {"s": t} if s["r"] is not None else {}
        if case["e4m3"]:
            # the 8-bit values follow the scale of 32 bits: only the scale itself has a value in 64
            return {**out, "y8": None, "scale": n.abs().max(1).values / E4M3_MAX}
        return {**out, "y": n}
    if op == "norm_bwd":
        # through y = c / r, c = x - mean x, r = sqrt(mean c^2 + eps): dc = u / r - c <u, c> / (width r^3), dx = dc - mean dc
        c = d["x"] - d["x"].mean(1, keepdim=True)
        r = ((c ** 2).sum(1, keepdim=True) / case["width"] + EPS) ** 0.5
        u = d["dy"] * d["w"]
        dc = u / r - c * ((u * c).sum(1, keepdim=True) / (case["width"] * r ** 3))
        ds = dc - dc.mean(1, keepdim=True)
        out = {"ds": ds if s["dsum"] is None else ds + d["dsum"], "dweight": torch.einsum("ij,ij->j", d["dy"], c / r)}
        return {**out, "dbias": torch.einsum("ij->j", d["dy"])} if case["bias"] else out
    tokens = s["tokens"].long()
    if op == "embed":
        at = torch.where(tokens >= 0, tokens, 0)
        return torch.where((tokens >= 0)[:, None], torch.index_select(d["table"], 0, at) * case["scale"], 0.0)
    # sums over the sorted tokens' runs, one more row for the padding
    order = torch.argsort(tokens)
    t = torch.zeros(case["vocab"] + 1, case["width"], device=DEV, dtype=torch.float64)
    t.index_put_((torch.where(tokens >= 0, tokens, case["vocab"])[order],), d["dy"][order], accumulate=True)
    return t[:-1] * case["scale"]


def _exact_token(case, d, i, S):
    """The definition, head by head: S <- (I - beta k k^T) Diag(alpha) S + beta k v^T, o = scale S^T q."""
    H, G, n = case["H"], case["G"], case["d"]
    if case["v_first"]:
        S = S.transpose(1, 2)
    k, v, b = d["k"][i], d["v"][i], d["beta"][i][:, None, None]
    keep = torch.eye(n, device=S.device, dtype=S.dtype) - b * torch.einsum("hi,hj->hij", k, k)
    S = torch.einsum("hij,hjv->hiv", keep, torch.exp(d["g"][i]).reshape(H, -1, 1) * S) + b * torch.einsum("hk,hv->hkv", k, v)
    o = torch.einsum("hgk,hkv->hgv", d["q"][i].reshape(H, G, n), S).reshape(H * G, n) * n ** -0.5
    return o, S.transpose(1, 2) if case["v_first"] else S
