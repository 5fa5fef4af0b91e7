"""The layer steps around the token mixers, as cases that can be timed and compared.

Three operators, each in its directions and types: the gated linear
recurrence (forward, backward, one-token step), the RMS norm with the
residual's addition (16 / 32-bit and e4m3 outputs, backward) and the matrix
product with bias, activation and residual (bf16, e4m3, backward).  ``run``
computes a case with elementary torch operations (``own`` false) or through
``context_merge_gb300.cpdr.Context`` (``own`` true); ``exact`` computes it in
64 bits from the definition.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
GROUP = 16            # tokens between two kept states of the recurrence's carry
E4M3_MAX = 448.0
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # decoding a batch of 8: the norm before a projection, one launch, latency counts
        dict(name="norm_step_r8_w2048", op="norm", dtype="bf16", rows=8, width=2048, residual=True, e4m3=False),
        # prefill of 32768 tokens at 32 heads x 128: the norm whose 8-bit output an e4m3 projection reads
        dict(name="norm_e4m3_r32768_w4096", op="norm", dtype="bf16", rows=32768, width=4096, residual=True, e4m3=True),
        # norm of every head's output (128 wide) in fp32, an odd number of rows
        dict(name="norm_heads_fp32_r524289_w128", op="norm", dtype="fp32", rows=524289, width=128, residual=False,
             e4m3=False),
        # training: the norm's gradients, an odd number of rows, with the residual stream's gradient added
        dict(name="norm_bwd_r65535_w2048", op="norm_bwd", dtype="bf16", rows=65535, width=2048, dsum=True),
        # decoding a batch of 16: the q, k, v projections (3 x 16 heads x 128), bound by the weights
        dict(name="linear_step_m16_k2048_n6144", op="linear", e4m3=False, rows=16, K=2048, N=6144, act="silu",
             bias=True, residual=False),
        # prefill: the q, k, v projections of 32768 tokens from the norm's 8-bit output
        dict(name="linear_e4m3_m32768_k2048_n6144", op="linear", e4m3=True, rows=32768, K=2048, N=6144, act="none",
             bias=False, residual=False),
        # the output projection of 32 heads, with bias, GELU and the residual, an odd number of tokens
        dict(name="linear_gelu_m8191_k4096_n2048", op="linear", e4m3=False, rows=8191, K=4096, N=2048, act="gelu",
             bias=True, residual=True),
        # training: gradients of input, weight and bias of the q, k, v projections
        dict(name="linear_bwd_m16384_k2048_n6144", op="linear_bwd", rows=16384, K=2048, N=6144, act="silu"),
        # decoding a batch of 61 sequences and 3 empty rows over a pool of state slots
        dict(name="glr_step_n64_c4096", op="glr_step", dtype="bf16", rows=64, channels=4096, slots=256, empty=3),
        # one sequence of 262144 tokens at 16 heads x 128, final state kept, ready for a backward
        dict(name="glr_t262144_c2048", op="glr", dtype="bf16", T=262144, seqs=1, channels=2048, zigzag=0, h0=False,
             carry=True),
        # a packed batch of 12 ragged sequences in fp32, zigzag order of 8 ranks, from initial states
        dict(name="glr_fp32_varlen65536_n12_c2048", op="glr", dtype="fp32", T=65536, seqs=12, channels=2048, zigzag=8,
             h0=True, carry=False),
        # training: gradients over a packed batch of 12 ragged sequences
        dict(name="glr_bwd_varlen65536_n12_c2048", op="glr_bwd", dtype="bf16", T=65536, seqs=12, channels=2048,
             zigzag=0, h0=True),
    ]


def _log(rng, lo, hi, mult=1):
    x = math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999 * mult)))
    return max(lo, min(hi, int(x) // mult * mult))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_bwd", "linear", "linear", "linear_bwd", "glr_step", "glr", "glr", "glr_bwd"])
    if op in ("norm", "norm_bwd"):
        width = rng.choice([128, _log(rng, 8, 8192, 8), _log(rng, 1024, 16384, 8)])
        rows = _log(rng, 1, max(2, (1 << 27) // width))
        if op == "norm_bwd":
            return dict(op=op, dtype=rng.choice(["bf16", "bf16", "fp32"]), rows=rows, width=width,
                        dsum=rng.random() < 0.5)
        e4m3 = rng.random() < 0.4
        return dict(op=op, dtype="bf16" if e4m3 else rng.choice(["bf16", "fp32"]), rows=rows, width=width,
                    residual=rng.random() < 0.6, e4m3=e4m3)
    if op in ("linear", "linear_bwd"):
        K, N = _log(rng, 64, 8192, 16), _log(rng, 64, 8192, 8)
        rows = _log(rng, 1, max(2, min(32768, (1 << (38 if op == "linear" else 37)) // (K * N))))
        act = rng.choice(["none", "silu", "gelu"])
        if op == "linear_bwd":
            return dict(op=op, rows=rows, K=K, N=N, act=act)
        return dict(op=op, e4m3=rng.random() < 0.4, rows=rows, K=K, N=N, act=act, bias=rng.random() < 0.6,
                    residual=rng.random() < 0.5)
    if op == "glr_step":
        rows = _log(rng, 1, 512)
        return dict(op=op, dtype=rng.choice(["bf16", "fp32"]), rows=rows, channels=_log(rng, 64, 8192, 8),
                    slots=rows + rng.randrange(0, 257), empty=rng.randrange(0, max(1, rows // 4)))
    C = _log(rng, 64, 4096, 8)
    zigzag = rng.choice([0, 0, 1, 2, 8])
    T = _log(rng, 1, min(131072, (1 << 27) // C))
    if zigzag:
        T = max(1, T // (2 * zigzag)) * 2 * zigzag
    return dict(op=op, dtype=rng.choice(["bf16", "bf16", "fp32"]), T=T, seqs=rng.choice([1, min(T, 1 + rng.randrange(40))]),
                channels=C, zigzag=zigzag, h0=rng.random() < 0.5,
                **({"carry": rng.random() < 0.5} if op == "glr" else {}))


# ------------------------------------------------------------------ inputs
def _lengths(T, n):
    """n ragged lengths of at least one token that sum to T (a fixed function of T and n)."""
    w = [1.0 + 3.0 * ((7 * i * i + 3 * i + 5) % 11) / 11.0 for i in range(n)]
    cuts = [0]
    for i in range(n):
        left = n - 1 - i
        want = cuts[-1] + max(1, int(w[i] * T / sum(w)))
        cuts.append(T if left == 0 else min(want, T - left))
    return cuts


def _order(T, R):
    """Memory position of every sequence position: zigzag order of R ranks (2R parts), identity for R = 0."""
    if not R:
        return None
    L = T // (2 * R)
    slot = torch.tensor([2 * r if r < R else 2 * (2 * R - 1 - r) + 1 for r in range(2 * R)], device=DEV)
    return (slot[:, None] * L + torch.arange(L, device=DEV)[None, :]).reshape(-1)


def _seq(state, x):
    """x [T, C] brought to sequence order."""
    return x if state["order"] is None else x[state["order"]]


def _mem(state, x):
    """x [T, C] put back in memory order."""
    if state["order"] is None:
        return x
    out = torch.empty_like(x)
    out[state["order"]] = x
    return out


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device=DEV)

    op = case["op"]
    s = {"case": case}
    if op in ("norm", "norm_bwd"):
        rows, width, dt = case["rows"], case["width"], DTYPES[case["dtype"]]
        x = randn(rows, width)
        x *= torch.exp(0.5 * randn(rows, 1))       # rows of differing size, as a residual stream has
        s["x"] = x.to(dt)
        s["w"] = 1.0 + 0.2 * randn(width)
        if op == "norm":
            if case["residual"]:
                s["r"] = randn(rows, width).to(dt)
        else:
            s["dy"] = randn(rows, width).to(dt)
            if case["dsum"]:
                s["dsum"] = randn(rows, width).to(dt)
    elif op in ("linear", "linear_bwd"):
        M, K, N = case["rows"], case["K"], case["N"]
        w = randn(N, K) / math.sqrt(K)
        if op == "linear" and case["e4m3"]:
            x = randn(M, K)
            for t, name in ((x, "x"), (w, "w")):
                scale = t.abs().amax(dim=1) / E4M3_MAX
                s[name] = (t / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
                s[name + "s"] = scale
        else:
            s["x"], s["w"] = randn(M, K).bfloat16(), w.bfloat16()
        if op == "linear":
            s["b"] = 0.1 * randn(N) if case["bias"] else None
            s["r"] = randn(M, N).bfloat16() if case["residual"] else None
        else:
            s["dy"] = randn(M, N).bfloat16()
            s["z"] = randn(M, N).bfloat16() if case["act"] != "none" else None
    elif op == "glr_step":
        n, C, S, dt = case["rows"], case["channels"], case["slots"], DTYPES[case["dtype"]]
        s["x"] = randn(n, C).to(dt)
        s["g"] = torch.nn.functional.logsigmoid(4.0 + 0.5 * randn(n, C))
        s["state"] = 4.0 * randn(S, C)
        slots = torch.randperm(S, generator=gen, device=DEV)[:n].to(torch.int32)
        empty = torch.randperm(n, generator=gen, device=DEV)[:case["empty"]]
        slots[empty] = -1
        s["slots"] = slots
        s["live"] = torch.nonzero(slots >= 0)[:, 0]
        s["y"] = torch.zeros(n, C, device=DEV, dtype=dt)
        s["state_out"] = s["state"].clone()
    else:
        T, C, n, dt = case["T"], case["channels"], case["seqs"], DTYPES[case["dtype"]]
        s["x"] = randn(T, C).to(dt)
        s["g"] = torch.nn.functional.logsigmoid(4.0 + 0.5 * randn(T, C))
        s["cuts"] = _lengths(T, n)
        s["starts"] = torch.tensor(s["cuts"][:-1], device=DEV)
        s["ends"] = torch.tensor(s["cuts"][1:], device=DEV) - 1
        s["longest"] = max(b - a for a, b in zip(s["cuts"], s["cuts"][1:]))
        s["order"] = _order(T, case["zigzag"])
        s["h0"] = 4.0 * randn(n, C) if case["h0"] else None
        if op == "glr_bwd":
            s["dy"] = randn(T, C).to(dt)
            s["dhT"] = randn(n, C)
            # the states that a training forward keeps: before every GROUP-th token of each sequence
            h = _prev(s, _scan(s, *_plain_ab(s)))
            at = torch.cat([torch.arange(a, b, GROUP) for a, b in zip(s["cuts"], s["cuts"][1:])])
            s["carry"] = h[at.to(DEV)].contiguous()
    if own:
        _prepare_own(s)
    return s


def _prepare_own(s):
    """The context, workspaces and output buffers that a user's program keeps between calls."""
    from context_merge_gb300 import cpdr

    case, op = s["case"], s["case"]["op"]
    f32 = torch.float32
    if op.startswith("glr") and op != "glr_step":
        T, C, R = case["T"], case["channels"], max(1, case["zigzag"])
        ctx = s["ctx"] = cpdr.Context(1, T, 1, 64, R, dtype=case["dtype"], cu_seqlens=s["cuts"],
                                      layout="zigzag" if case["zigzag"] else "contiguous")
        for k in ("x", "g", "dy"):
            if k in s:
                s[k] = s[k].view(1, T, C)
        if op == "glr":
            s["y"] = torch.empty_like(s["x"])
            s["hT"] = torch.empty(case["seqs"], C, device=DEV, dtype=f32)
            s["carry"] = torch.empty(ctx.glr_carry_shape(C), device=DEV, dtype=f32) if case["carry"] else None
        else:
            s["out"] = dict(dx=torch.empty_like(s["x"]), dg=torch.empty_like(s["g"]),
                            dh0=torch.empty(case["seqs"], C, device=DEV, dtype=f32))
        return
    ctx = s["ctx"] = cpdr.Context(1, 1, 1, 64, 1, dtype=case.get("dtype", "bf16"))
    if op == "norm":
        x = s["x"]
        s["s"] = torch.empty_like(x) if case["residual"] else None
        s["y"] = None if case["e4m3"] else torch.empty_like(x)
        s["y8"] = torch.empty(x.shape, device=DEV, dtype=torch.float8_e4m3fn) if case["e4m3"] else None
        s["ys"] = torch.empty(x.shape[0], device=DEV, dtype=f32) if case["e4m3"] else None
    elif op == "norm_bwd":
        s["out"] = dict(ds=torch.empty_like(s["x"]), dweight=torch.empty_like(s["w"]))
        s["ws"] = torch.empty(ctx.rmsnorm_bwd_workspace_bytes(case["rows"], case["width"]), device=DEV, dtype=torch.uint8)
    elif op == "linear":
        s["y"] = torch.empty(case["rows"], case["N"], device=DEV, dtype=torch.bfloat16)
    elif op == "linear_bwd":
        s["out"] = dict(dx=torch.empty_like(s["x"]), dw=torch.empty_like(s["w"]),
                        dbias=torch.empty(case["N"], device=DEV, dtype=f32))
        s["ws"] = torch.empty(ctx.linear_bwd_workspace_bytes(case["rows"], case["K"], case["N"], case["act"]),
                              device=DEV, dtype=torch.uint8)


# ------------------------------------------------------------------ one pass
def run(state):
    op = state["case"]["op"]
    return (_OWN if own else _PLAIN)[op](state)


def _own_norm(s):
    s["ctx"].rmsnorm_fwd(s["x"], s["w"], residual=s.get("r"), sum_out=s["s"], y=s["y"], y8=s["y8"], scale=s["ys"], eps=EPS)
    out = {"y8": s["y8"], "scale": s["ys"]} if s["case"]["e4m3"] else {"y": s["y"]}
    if s["s"] is not None:
        out["s"] = s["s"]
    return out


def _own_norm_bwd(s):
    return s["ctx"].rmsnorm_bwd(s["x"], s["w"], s["dy"], dsum=s.get("dsum"), eps=EPS, out=s["out"], workspace=s["ws"])


def _own_linear(s):
    s["ctx"].linear_fwd(s["x"], s["w"], s["y"], bias=s["b"], activation=s["case"]["act"], residual=s["r"],
                        x_scale=s.get("xs"), w_scale=s.get("ws"))
    return s["y"]


def _own_linear_bwd(s):
    return s["ctx"].linear_bwd(s["x"], s["w"], s["dy"], z=s["z"], activation=s["case"]["act"], out=s["out"], workspace=s["ws"])


def _own_glr_step(s):
    s["ctx"].glr_step(s["x"], s["g"], s["state"], s["y"], slots=s["slots"], state_out=s["state_out"])
    return {"y": s["y"], "state": s["state_out"]}


def _own_glr(s):
    s["ctx"].glr_fwd(s["x"], s["g"], s["y"], h0=s["h0"], hT=s["hT"], carry=s["carry"])
    return {"y": s["y"][0], "hT": s["hT"]}


def _own_glr_bwd(s):
    r = s["ctx"].glr_bwd(s["x"], s["g"], s["carry"], s["dy"], dhT=s["dhT"], out=s["out"])
    return {"dx": r["dx"][0], "dg": r["dg"][0], "dh0": r["dh0"]}


_OWN = dict(norm=_own_norm, norm_bwd=_own_norm_bwd, linear=_own_linear, linear_bwd=_own_linear_bwd,
            glr_step=_own_glr_step, glr=_own_glr, glr_bwd=_own_glr_bwd)


def _plain_norm(s):
    t = s["x"].float()
    out = {}
    if "r" in s:
        t = t + s["r"].float()
        out["s"] = t.to(s["x"].dtype)
    n = t * torch.rsqrt((t * t).mean(dim=1, keepdim=True) + EPS) * s["w"]
    if s["case"]["e4m3"]:
        scale = (n.abs().amax(dim=1) / E4M3_MAX).clamp(min=2.0 ** -126)
        out["y8"] = (n / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        out["scale"] = scale
    else:
        out["y"] = n.to(s["x"].dtype)
    return out


def _plain_norm_bwd(s):
    t, dy = s["x"].float(), s["dy"].float()
    rstd = torch.rsqrt((t * t).mean(dim=1, keepdim=True) + EPS)
    xh = t * rstd
    wdy = dy * s["w"]
    ds = rstd * (wdy - xh * (wdy * xh).mean(dim=1, keepdim=True))
    if "dsum" in s:
        ds = ds + s["dsum"].float()
    return {"ds": ds.to(s["x"].dtype), "dweight": (dy * xh).sum(dim=0)}


def _act(z, act):
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    return z


def _act_grad(z, act):
    if act == "silu":
        sg = 1.0 / (1.0 + torch.exp(-z))
        return sg * (1.0 + z * (1.0 - sg))
    return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)


def _plain_linear(s):
    z = s["x"].float() @ s["w"].float().t()
    if s["case"]["e4m3"]:
        z = z * s["xs"][:, None] * s["ws"]
    if s["b"] is not None:
        z = z + s["b"]
    y = _act(z, s["case"]["act"])
    if s["r"] is not None:
        y = y + s["r"].float()
    return y.bfloat16()


def _plain_linear_bwd(s):
    dz = s["dy"].float()
    if s["z"] is not None:
        dz = dz * _act_grad(s["z"].float(), s["case"]["act"])
    return {"dx": (dz @ s["w"].float()).bfloat16(), "dw": (dz.t() @ s["x"].float()).bfloat16(), "dbias": dz.sum(dim=0)}


def _plain_glr_step(s):
    live = s["live"]
    at = s["slots"][live].long()
    h = torch.exp(s["g"][live]) * s["state"][at] + s["x"][live].float()
    s["state_out"][at] = h
    s["y"][live] = h.to(s["y"].dtype)
    return {"y": s["y"], "state": s["state_out"]}


def _plain_ab(s):
    """The recurrence's factors and terms in sequence order, initial states folded into the first tokens."""
    a, b = torch.exp(_seq(s, s["g"])), _seq(s, s["x"]).float().clone()
    if s["h0"] is not None:
        b[s["starts"]] += a[s["starts"]] * s["h0"]
    return a.index_fill(0, s["starts"], 0.0), b


def _scan(s, a, b):
    """h_t = a_t h_{t-1} + b_t over the rows, by doubling (a is zero at each sequence's first token)."""
    step = 1
    while step < s["longest"]:
        b[step:] = b[step:] + a[step:] * b[:-step]
        a[step:] = a[step:] * a[:-step]
        step *= 2
    return b


def _prev(s, h):
    """The state before each token."""
    p = torch.roll(h, 1, 0)
    p[s["starts"]] = 0.0 if s["h0"] is None else s["h0"]
    return p


def _plain_glr(s):
    h = _scan(s, *_plain_ab(s))
    return {"y": _mem(s, h.to(s["x"].dtype)), "hT": h[s["ends"]]}


def _plain_glr_bwd(s):
    p = _prev(s, _scan(s, *_plain_ab(s)))
    a, dh = torch.exp(_seq(s, s["g"])), _seq(s, s["dy"]).float().clone()
    dh[s["ends"]] += s["dhT"]
    nxt = torch.roll(a, -1, 0).index_fill(0, s["ends"], 0.0)
    dh = _scan(s, nxt.flip(0), dh.flip(0)).flip(0)
    return {"dx": _mem(s, dh.to(s["x"].dtype)), "dg": _mem(s, dh * a * p), "dh0": (a * dh)[s["starts"]]}


_PLAIN = dict(norm=_plain_norm, norm_bwd=_plain_norm_bwd, linear=_plain_linear, linear_bwd=_plain_linear_bwd,
              glr_step=_plain_glr_step, glr=_plain_glr, glr_bwd=_plain_glr_bwd)


# ------------------------------------------------------------------ work
def work(case):
    op = case["op"]
    es = 4 if case.get("dtype") == "fp32" else 2
    if op == "norm":
        n = case["rows"] * case["width"]
        return {"bytes": n * (es + (2 * es if case["residual"] else 0) + (1 if case["e4m3"] else es)) + 4 * case["width"]
                + (4 * case["rows"] if case["e4m3"] else 0), "flops": 5 * n}
    if op == "norm_bwd":
        n = case["rows"] * case["width"]
        return {"bytes": n * es * (4 if case["dsum"] else 3) + 8 * case["width"], "flops": 10 * n}
    if op == "linear":
        M, K, N = case["rows"], case["K"], case["N"]
        ei = 1 if case["e4m3"] else 2
        return {"bytes": ei * (M * K + N * K) + 2 * M * N * (2 if case["residual"] else 1) + (4 * N if case["bias"] else 0)
                + (4 * (M + N) if case["e4m3"] else 0), "flops": 2 * M * N * K}
    if op == "linear_bwd":
        M, K, N = case["rows"], case["K"], case["N"]
        return {"bytes": 4 * (M * K + N * K) + 2 * M * N * (1 if case["act"] == "none" else 2) + 4 * N,
                "flops": 4 * M * N * K}
    if op == "glr_step":
        n = (case["rows"] - case["empty"]) * case["channels"]
        return {"bytes": n * (2 * es + 12) + 4 * case["rows"], "flops": 3 * n}
    n, m = case["T"] * case["channels"], case["seqs"] * case["channels"]
    if op == "glr":
        return {"bytes": n * (2 * es + 4) + (n * 4 // GROUP if case["carry"] else 0) + 4 * m * (2 if case["h0"] else 1),
                "flops": 3 * n}
    return {"bytes": n * (3 * es + 8) + n * 4 // GROUP + 8 * m, "flops": 8 * n}


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
    if op == "norm":
        t = d["x"] + d["r"] if "r" in d else d["x"]
        n = t / ((t ** 2).sum(1, keepdim=True) / case["width"] + EPS) ** 0.5 * d["w"]
        out = {"s": t} if "r" in d else {}
        if case["e4m3"]:
            # the 8-bit values follow the scale of 32 bits: only the scale itself has a value in 64
            return {**out, "y8": None, "scale": n.abs().max(1).values / E4M3_MAX}
        return {**out, "y": n}
    if op == "norm_bwd":
        # through the Jacobian of x -> x / r, r = sqrt(mean x^2 + eps)
        r = ((d["x"] ** 2).sum(1, keepdim=True) / case["width"] + EPS) ** 0.5
        u = d["dy"] * d["w"]
        ds = u / r - d["x"] * ((u * d["x"]).sum(1, keepdim=True) / (case["width"] * r ** 3))
        return {"ds": ds + d["dsum"] if "dsum" in d else ds, "dweight": (d["dy"] * d["x"] / r).sum(0)}
    if op == "linear":
        if 2.0 * case["rows"] * case["K"] * case["N"] > 4e12:
            return None
        z = torch.einsum("mk,nk->mn", d["x"], d["w"])
        if case["e4m3"]:
            z = torch.einsum("mn,m,n->mn", z, d["xs"], d["ws"])
        if s["b"] is not None:
            z = z + d["b"]
        if case["act"] == "silu":
            z = z * torch.sigmoid(z)
        elif case["act"] == "gelu":
            z = z * torch.special.ndtr(z)
        return z + d["r"] if s["r"] is not None else z
    if op == "linear_bwd":
        if 4.0 * case["rows"] * case["K"] * case["N"] > 4e12:
            return None
        dz = d["dy"]
        if case["act"] == "silu":
            p = torch.sigmoid(d["z"])
            dz = dz * (p + d["z"] * p * torch.sigmoid(-d["z"]))
        elif case["act"] == "gelu":
            pdf = torch.exp(-d["z"] ** 2 / 2) * (2 * math.pi) ** -0.5
            dz = dz * (torch.special.ndtr(d["z"]) + d["z"] * pdf)
        return {"dx": torch.einsum("mn,nk->mk", dz, d["w"]), "dw": torch.einsum("mn,mk->nk", dz, d["x"]),
                "dbias": torch.einsum("mn->n", dz)}
    if op == "glr_step":
        y, state = s["y"].double(), d["state_out"].clone()
        for i, slot in enumerate(s["slots"].tolist()):
            if slot >= 0:
                state[slot] = torch.exp(d["g"][i]) * d["state"][slot] + d["x"][i]
                y[i] = state[slot]
        return {"y": y, "state": state}
    # the recurrence token by token: every sequence is cut into pieces of up to LEN tokens, all pieces
    # step together from a zero state, and the pieces' starting states follow one another
    T, C, cuts, LEN = case["T"], case["channels"], s["cuts"], 512
    mem = _order(T, case["zigzag"])
    mem = torch.arange(T, device=DEV) if mem is None else mem
    a, x = torch.exp(d["g"][mem]), d["x"][mem]
    h0 = d["h0"] if s["h0"] is not None else torch.zeros(len(cuts) - 1, C, device=DEV, dtype=torch.float64)
    h, hT = _exact_scan(a, x, h0, cuts, LEN)
    if op == "glr":
        y = torch.empty_like(h)
        y[mem] = h
        return {"y": y, "hT": hT}
    prev = torch.cat([h[:1], h[:-1]])
    for n, c in enumerate(cuts[:-1]):
        prev[c] = h0[n]
    # in reverse: dh_t = dy_t + a_{t+1} dh_{t+1}, begun from dhT behind each sequence's last token
    after = torch.cat([a[1:], a[:1]])
    for c in cuts[1:]:
        after[c - 1] = 1.0
    back = [T - c for c in reversed(cuts)]
    dh, _ = _exact_scan(after.flip(0), d["dy"][mem].flip(0), d["dhT"].flip(0), back, LEN)
    dh = dh.flip(0)
    dx, dg = torch.empty_like(dh), torch.empty_like(dh)
    dx[mem], dg[mem] = dh, dh * a * prev
    first = torch.tensor(cuts[:-1], device=DEV)
    return {"dx": dx, "dg": dg, "dh0": a[first] * dh[first]}


def _exact_scan(a, x, h0, cuts, LEN):
    pieces = [(n, t, min(t + LEN, e)) for n, (c, e) in enumerate(zip(cuts, cuts[1:])) for t in range(c, e, LEN)]
    begin = torch.tensor([p[1] for p in pieces], device=x.device)
    end = torch.tensor([p[2] for p in pieces], device=x.device)
    h = torch.zeros_like(x)
    run_a = torch.ones(len(pieces), x.shape[1], device=x.device, dtype=x.dtype)
    run_h = torch.zeros_like(run_a)
    kept = torch.empty_like(a)            # product of a from the piece's first token on
    for i in range(max(e - b for _, b, e in pieces)):
        on = begin + i < end
        t = (begin + i)[on]
        run_h[on] = a[t] * run_h[on] + x[t]
        run_a[on] = run_a[on] * a[t]
        h[t], kept[t] = run_h[on], run_a[on]
    hT = h0.clone()
    for k, (n, b, e) in enumerate(pieces):
        h[b:e] += kept[b:e] * hT[n]
        hT[n] = h[e - 1]
    return h, hT
