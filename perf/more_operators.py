"""Cases that time what a sampler's layer does with the FP8 weights that the
receiver keeps, and the same operators in elementary torch operations.

  norm    root-mean-square norm, with the residual's addition in front of it; the output
          as E4M3 codes with a scale for each 128 columns of a row (serving), or as
          BF16 with the backward pass behind it (training)
  quant   a BF16 matrix, or silu(gate) * up of a [gate, up] matrix, as such codes and scales
  gemm    such rows times the weights that are held in 128 x 128 blocks ("nt": y = x W^T with
          an optional bias; "nn": dx = dy W, the gradient of x)
  moe     a mixture-of-experts layer for a few tokens: the router's choice from its
          logits, then each token's experts with their weights in 128 x 128 blocks
"""
import math

import torch

own = False  # False: elementary torch operations; True: the library's calls

GROUP = 128          # columns that share a scale; blocks of weights are GROUP x GROUP
TOP = 448.0          # the largest E4M3 value
TINY = 2.0 ** -96    # groups whose largest value is below are stored as zero
EPS = 1e-6


def listed():
    return [
        # the norm in front of a projection for one request's next token: latency alone
        {"name": "norm-one-token", "op": "norm", "tokens": 1, "hidden": 5120, "residual": True, "train": False},
        # the same for prompts, hidden size of the 32B-shaped set
        {"name": "norm-prefill", "op": "norm", "tokens": 8192, "hidden": 5120, "residual": True, "train": False},
        # a ragged training batch at the 8B-shaped set's hidden size: BF16 output, then dx and dweight
        {"name": "norm-train", "op": "norm", "tokens": 4099, "hidden": 4096, "residual": True, "train": True},
        # the MLP's activation of one token each of many requests, [gate, up] of the 32B-shaped set
        {"name": "glu-decode", "op": "quant", "tokens": 96, "cols": 27648, "glu": True},
        # a gradient on its way into the product that gives dx, the [gate, up] rows of the 8B-shaped set
        {"name": "quant-gradient", "op": "quant", "tokens": 8191, "cols": 28672, "glu": False},
        # one token through [q; k; v] of the 32B-shaped set, which has biases
        {"name": "gemm-one-token", "op": "gemm", "tokens": 1, "k": 5120, "n": 7168, "form": "nt", "bias": True},
        # one token each of many requests through the MLP's down projection
        {"name": "gemm-decode", "op": "gemm", "tokens": 96, "k": 27648, "n": 5120, "form": "nt", "bias": False},
        # prompts through [gate; up]
        {"name": "gemm-prefill", "op": "gemm", "tokens": 8192, "k": 5120, "n": 55296, "form": "nt", "bias": False},
        # adapters trained over the frozen FP8 weights: dx of [gate; up] of the 8B-shaped set
        {"name": "gemm-dx", "op": "gemm", "tokens": 4099, "k": 4096, "n": 28672, "form": "nn", "bias": False},
        # one token through the expert layer of hidden 7168: 8 of 384 experts
        {"name": "moe-one-token", "op": "moe", "tokens": 1, "hidden": 7168, "inter": 2048, "experts": 384, "top_k": 8},
        # one token each of many requests on small experts, odd counts
        {"name": "moe-ragged", "op": "moe", "tokens": 61, "hidden": 2048, "inter": 1408, "experts": 60, "top_k": 4},
        # few large experts, each with some dozens of the tokens
        {"name": "moe-few-experts", "op": "moe", "tokens": 256, "hidden": 4096, "inter": 14336, "experts": 16,
         "top_k": 2},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "quant", "gemm", "gemm", "gemm", "moe", "moe"])
    if op == "norm":
        train = rng.random() < 0.4
        return {"op": op, "tokens": _log_int(rng, 1, 8192), "hidden": 8 * _log_int(rng, 16, 1024),
                "residual": rng.random() < 0.6, "train": train}
    if op == "quant":
        return {"op": op, "tokens": _log_int(rng, 1, 8192), "cols": 16 * _log_int(rng, 8, 1700), "glu": rng.random() < 0.5}
    if op == "gemm":
        # single tokens and small batches half of the time
        tokens = _log_int(rng, 1, 128) if rng.random() < 0.5 else _log_int(rng, 129, 8192)
        form = rng.choice(["nt", "nt", "nn"])
        n = _log_int(rng, 100, 28000) if form == "nt" else 16 * _log_int(rng, 8, 1700)
        k = 16 * _log_int(rng, 8, 1700)
        return {"op": op, "tokens": min(tokens, 2 * 10 ** 12 // (n * k)), "k": k, "n": n, "form": form,
                "bias": form == "nt" and rng.random() < 0.3}
    hidden, inter = 16 * _log_int(rng, 16, 448), 16 * _log_int(rng, 8, 256)
    experts = min(_log_int(rng, 4, 256), 3 * 10 ** 9 // (3 * hidden * inter))
    return {"op": op, "tokens": _log_int(rng, 1, 256), "hidden": hidden, "inter": inter, "experts": experts,
            "top_k": rng.randint(1, min(8, experts))}


def _up(n, m=GROUP):
    return -(-n // m)


def work(case):
    t = case["tokens"]
    if case["op"] == "norm":
        h, res = case["hidden"], case["residual"]
        if case["train"]:
            # x and stream read, stream and y written; stream, dy and its own gradient read, dx written
            return {"bytes": t * h * ((4 if res else 0) + 4 + 6 + (2 if res else 0)) + 8 * h, "flops": 16 * t * h}
        return {"bytes": t * h * (2 + (4 if res else 0) + 1) + 4 * t * _up(h) + 2 * h, "flops": 8 * t * h}
    if case["op"] == "quant":
        c = case["cols"]
        return {"bytes": t * c * (5 if case["glu"] else 3) + 4 * t * _up(c), "flops": (10 if case["glu"] else 4) * t * c}
    if case["op"] == "gemm":
        k, n = case["k"], case["n"]
        inner, out = (k, n) if case["form"] == "nt" else (n, k)
        return {"bytes": k * n + 4 * _up(k) * _up(n) + t * inner + 4 * t * _up(inner) + 2 * t * out, "flops": 2 * t * k * n}
    h, i, e, top = case["hidden"], case["inter"], case["experts"], case["top_k"]
    used = e * (1 - (1 - top / e) ** t)  # experts with a token, on average
    return {"bytes": int(used * 3 * h * i + 4 * t * h + 4 * t * e + 12 * t * top), "flops": 6 * t * top * h * i}


# ---- inputs ------------------------------------------------------------------------
def _weights(gen, shape):
    """Codes and block scales of weights about as large as 1 / sqrt(columns): the largest of a
    block's 16384 normal values lies about 4.2 deviations out and has the largest code."""
    codes = torch.empty(shape, dtype=torch.uint8, device="cuda")
    flat = codes.view(-1)
    for at in range(0, flat.numel(), 1 << 28):
        part = flat[at:at + (1 << 28)]
        z = torch.empty(part.numel(), device="cuda").normal_(0.0, TOP / 4.2, generator=gen).clamp_(-TOP, TOP)
        part.copy_(z.to(torch.float8_e4m3fn).view(torch.uint8))
    blocks = (*shape[:-2], _up(shape[-2]), _up(shape[-1]))
    scales = torch.empty(blocks, device="cuda").uniform_(0.9, 1.1, generator=gen).mul_(4.2 / TOP / math.sqrt(shape[-1]))
    return codes, scales


def _rows_quantised(x):
    """Codes and scales of the rows of x in groups of 128 columns, as a norm leaves them."""
    t, c = x.shape
    g = torch.nn.functional.pad(x, (0, -c % GROUP)).view(t, -1, GROUP)
    scales = g.abs().amax(2) / TOP
    codes = (g / scales[:, :, None]).to(torch.float8_e4m3fn).view(t, -1)[:, :c]
    return codes.contiguous().view(torch.uint8), scales


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    bf16 = torch.bfloat16

    def normal(shape, std, dtype=bf16):
        return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=gen)

    st = {"case": dict(case)}
    t, op = case["tokens"], case["op"]
    if op == "norm":
        h = case["hidden"]
        st["x"], st["weight"] = normal((t, h), 0.7), 1 + normal((h,), 0.01)
        # a residual stream has a few columns that are much larger than the others
        st["residual"] = normal((t, h), 1.5) if case["residual"] else None
        if case["residual"]:
            st["residual"][:, ::509] *= 20
        if case["train"]:
            st["dy"] = normal((t, h), 1e-2)
            st["dres"] = normal((t, h), 1e-2) if case["residual"] else None
            for name in ("y", "dx"):
                st[name] = torch.zeros((t, h), dtype=bf16, device="cuda")
            st["dweight"], st["rstd"] = torch.zeros(h, device="cuda"), torch.zeros(t, device="cuda")
        else:
            st["codes"] = torch.zeros((t, h), dtype=torch.uint8, device="cuda")
            st["scales"] = torch.zeros((t, _up(h)), device="cuda")
        if own and case["train"]:
            import sparse_delta_codec_amd as pulse

            st["ws"] = pulse.rms_norm_workspace(t, h)
    elif op == "quant":
        c = case["cols"]
        st["x"] = normal((t, 2 * c), 1.5) if case["glu"] else normal((t, c), 1e-2)
        st["codes"] = torch.zeros((t, c), dtype=torch.uint8, device="cuda")
        st["scales"] = torch.zeros((t, _up(c)), device="cuda")
    elif op == "gemm":
        k, n = case["k"], case["n"]
        inner, out = (k, n) if case["form"] == "nt" else (n, k)
        st["w"], st["w_scales"] = _weights(gen, (n, k))
        st["x"], st["x_scales"] = _rows_quantised(normal((t, inner), 1.0, torch.float32))
        st["bias"] = normal((n,), 0.5) if case["bias"] else None
        st["y"] = torch.zeros((t, out), dtype=bf16, device="cuda")
        if own:
            import sparse_delta_codec_amd as pulse

            st["ws"] = pulse.fp8_gemm_workspace(t, n, k, form=case["form"])
    else:
        h, i, e, top = (case[x] for x in ("hidden", "inter", "experts", "top_k"))
        st["up"], st["up_scales"] = _weights(gen, (e, 2 * i, h))        # [gate; up] of every expert
        st["down"], st["down_scales"] = _weights(gen, (e, h, i))
        st["x"], st["logits"] = normal((t, h), 1.0), normal((t, e), 1.5, torch.float32)
        st["ids"] = torch.zeros((t, top), dtype=torch.int32, device="cuda")
        st["weights"] = torch.zeros((t, top), device="cuda")
        st["y"] = torch.zeros((t, h), dtype=bf16, device="cuda")
        if own:
            import sparse_delta_codec_amd as pulse

            st["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
            st["ws"] = pulse.moe_workspace(t, h, i, e, top)
    return st


# ---- the operators in elementary operations ------------------------------------------
def _to_codes(x, codes, scales):
    t, c = x.shape
    g = torch.nn.functional.pad(x, (0, -c % GROUP)).view(t, -1, GROUP)
    amax = g.abs().amax(2)
    live = amax >= TINY
    scales.copy_(torch.where(live, amax / TOP, torch.ones_like(amax)))
    q = torch.where(live[:, :, None], g / scales[:, :, None], torch.zeros_like(g))
    codes.copy_(q.to(torch.float8_e4m3fn).view(t, -1)[:, :c].view(torch.uint8))


def _norm(st):
    case, w = st["case"], st["weight"].float()
    stream = st["x"]
    if case["residual"]:  # the sum is what later layers and the backward pass read: rounded first
        st["residual"].copy_(st["x"].float() + st["residual"].float())
        stream = st["residual"]
    s = stream.float()
    rstd = torch.rsqrt(s.square().mean(1) + EPS)
    hat = s * rstd[:, None]
    out = {"residual": st["residual"]} if case["residual"] else {}
    if not case["train"]:
        _to_codes(hat * w, st["codes"], st["scales"])
        return out | {"codes": st["codes"].view(torch.float8_e4m3fn), "scales": st["scales"]}
    st["y"].copy_(hat * w)
    dy = st["dy"].float()
    st["dweight"].copy_((dy * hat).sum(0))
    g = dy * w
    dx = (g - hat * (g * hat).mean(1, keepdim=True)) * rstd[:, None]
    st["dx"].copy_(dx + st["dres"].float() if case["residual"] else dx)
    return out | {"y": st["y"], "dx": st["dx"], "dweight": st["dweight"]}


def _quant(st):
    x = st["x"].float()
    if st["case"]["glu"]:
        gate, up = x.chunk(2, dim=1)
        x = gate / (1 + torch.exp(-gate)) * up
    _to_codes(x, st["codes"], st["scales"])
    return {"codes": st["codes"].view(torch.float8_e4m3fn), "scales": st["scales"]}


def _block_values(codes, scales):
    """The values of a matrix in 128 x 128 blocks, in 32 bits."""
    n, k = codes.shape
    full = scales.repeat_interleave(GROUP, 0)[:n].repeat_interleave(GROUP, 1)[:, :k]
    return codes.view(torch.float8_e4m3fn).float() * full


def _gemm(st):
    x = st["x"].view(torch.float8_e4m3fn).float()
    x = x * st["x_scales"].repeat_interleave(GROUP, 1)[:, :x.shape[1]]
    w = _block_values(st["w"], st["w_scales"])
    y = x @ w.t() if st["case"]["form"] == "nt" else x @ w
    st["y"].copy_(y + st["bias"].float() if st["case"]["bias"] else y)
    return {"y": st["y"]}


def _moe(st):
    top = st["case"]["top_k"]
    # the largest logits, equal ones by the lowest index
    order = torch.sort(st["logits"], dim=1, descending=True, stable=True)
    st["ids"].copy_(order.indices[:, :top])
    st["weights"].copy_(torch.softmax(order.values[:, :top], 1))
    y = torch.zeros(st["y"].shape, device="cuda")
    for e in torch.unique(st["ids"]).tolist():
        rows, place = (st["ids"] == e).nonzero(as_tuple=True)
        gate, up = (st["x"][rows].float() @ _block_values(st["up"][e], st["up_scales"][e]).t()).chunk(2, dim=1)
        h = gate / (1 + torch.exp(-gate)) * up
        part = h @ _block_values(st["down"][e], st["down_scales"][e]).t()
        y[rows] += part * st["weights"][rows, place][:, None]
    st["y"].copy_(y)
    return {"ids": st["ids"], "weights": st["weights"], "y": st["y"]}


def _own(st):
    import sparse_delta_codec_amd as pulse

    case, op = st["case"], st["case"]["op"]
    if op == "norm":
        out = {"residual": st["residual"]} if case["residual"] else {}
        if not case["train"]:
            pulse.pulse_rms_norm(st["x"], st["weight"], eps=EPS, residual=st["residual"], codes=st["codes"],
                                 scales=st["scales"])
            return out | {"codes": st["codes"].view(torch.float8_e4m3fn), "scales": st["scales"]}
        pulse.pulse_rms_norm(st["x"], st["weight"], eps=EPS, residual=st["residual"], y=st["y"], rstd=st["rstd"])
        pulse.pulse_rms_norm_backward(st["residual"] if case["residual"] else st["x"], st["weight"], st["rstd"],
                                      st["dy"], st["dx"], st["dweight"], st["ws"], dres=st["dres"])
        return out | {"y": st["y"], "dx": st["dx"], "dweight": st["dweight"]}
    if op == "quant":
        pulse.fp8_group_quant(st["x"], st["codes"], st["scales"], glu=case["glu"])
        return {"codes": st["codes"].view(torch.float8_e4m3fn), "scales": st["scales"]}
    if op == "gemm":
        pulse.fp8_block_gemm(st["x"], st["x_scales"], st["w"], st["w_scales"], st["y"], st["ws"], bias=st["bias"],
                             form=case["form"])
        return {"y": st["y"]}
    pulse.pulse_moe_route(st["logits"], st["ids"], st["weights"])
    pulse.pulse_moe_forward(st["x"], st["ids"], st["weights"], st["up"], st["up_scales"], st["down"],
                            st["down_scales"], st["y"], st["status"], st["ws"])
    return {"ids": st["ids"], "weights": st["weights"], "y": st["y"]}


def run(state):
    if own:
        return _own(state)
    return {"norm": _norm, "quant": _quant, "gemm": _gemm, "moe": _moe}[state["case"]["op"]](state)


# ---- the definitions in 64 bits ------------------------------------------------------
def _exact_quantised(x):
    """Scales, and the quotients before they are rounded to E4M3."""
    t, c = x.shape
    quotients, scales = torch.empty_like(x), []
    for at in range(0, c, GROUP):
        part = x[:, at:at + GROUP]
        scale = part.abs().max(1).values / TOP
        scales.append(torch.where(scale * TOP < TINY, torch.ones_like(scale), scale))
        quotients[:, at:at + GROUP] = part / scales[-1][:, None]
    return {"codes": quotients, "scales": torch.stack(scales, 1)}


def _e4m3_table():
    """The value of every E4M3 code (the two codes that are no numbers do not occur)."""
    v = [(c & 7) / 8 * 2.0 ** -6 if c < 8 else (1 + (c & 7) / 8) * 2.0 ** ((c >> 3) - 7) for c in range(127)] + [math.nan]
    return torch.tensor(v + [-x for x in v], dtype=torch.float64, device="cuda")


def _exact_blocks(codes, scales):
    out = _e4m3_table()[codes.int()]
    for r in range(scales.shape[0]):
        for c in range(scales.shape[1]):
            out[r * GROUP:(r + 1) * GROUP, c * GROUP:(c + 1) * GROUP] *= scales[r, c].double()
    return out


def _exact_norm(case, st):
    out, w, n = {}, st["weight"].double(), case["hidden"]
    s = st["x"].double()
    if case["residual"]:
        out["residual"] = s + st["residual"].double()
        s = out["residual"].to(torch.bfloat16).double()  # the definition rounds the stream here
    rms = ((s * s).sum(1, keepdim=True) / n + EPS).sqrt()
    y = s / rms * w
    if not case["train"]:
        return out | _exact_quantised(y)
    dy = st["dy"].double()
    # y_j = w_j s_j / rms, d rms / d s_i = s_i / (n rms)
    along = (dy * w * s).sum(1, keepdim=True) / n
    dx = dy * w / rms - s * along / rms ** 3
    if case["residual"]:
        dx = dx + st["dres"].double()
    return out | {"y": y, "dx": dx, "dweight": (dy * s / rms).sum(0)}


def _exact_moe(case, st):
    top, y = case["top_k"], torch.zeros(st["y"].shape, dtype=torch.float64, device="cuda")
    logits, ids, weights = st["logits"].tolist(), [], []
    for row in logits:
        chosen = sorted(range(len(row)), key=lambda e: (-row[e], e))[:top]
        shares = [math.exp(row[e] - row[chosen[0]]) for e in chosen]
        ids.append(chosen)
        weights.append([s / math.fsum(shares) for s in shares])
    for e in sorted({e for chosen in ids for e in chosen}):
        mine = [(t, ids[t].index(e)) for t in range(case["tokens"]) if e in ids[t]]
        rows = torch.tensor([t for t, _ in mine], device="cuda")
        share = torch.tensor([weights[t][p] for t, p in mine], dtype=torch.float64, device="cuda")
        both = torch.mm(st["x"][rows].double(), _exact_blocks(st["up"][e], st["up_scales"][e]).t())
        gate, up = both[:, :case["inter"]], both[:, case["inter"]:]
        h = gate * torch.sigmoid(gate) * up
        y[rows] += share[:, None] * torch.mm(h, _exact_blocks(st["down"][e], st["down_scales"][e]).t())
    return {"ids": torch.tensor(ids, dtype=torch.int32), "weights": torch.tensor(weights, dtype=torch.float64), "y": y}


def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "norm":
        return _exact_norm(case, st)
    if case["op"] == "quant":
        x = st["x"].double()
        if case["glu"]:
            c = case["cols"]
            x = x[:, :c] * torch.sigmoid(x[:, :c]) * x[:, c:]
        return _exact_quantised(x)
    if case["op"] == "gemm":
        x, w = _e4m3_table()[st["x"].int()], _exact_blocks(st["w"], st["w_scales"])
        for g in range(st["x_scales"].shape[1]):
            x[:, g * GROUP:(g + 1) * GROUP] *= st["x_scales"][:, g:g + 1].double()
        y = torch.mm(x, w.t() if case["form"] == "nt" else w)
        return {"y": y + st["bias"].double() if case["bias"] else y}
    return _exact_moe(case, st)
