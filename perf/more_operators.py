"""More projections of a feed-forward sub-layer, as cases to be timed and compared: in 8-bit integers, and by expert.

  quantize   rows to 8 bits: scale = max |x| / 127 for each row, codes = x * (127 / max |x|) to the nearest (ties to even)
  linear8    out = act(xs[m] ws[n] sum over k of x[m, k] w[n, k] + bias) + residual, x and w codes in 8 bits
  gated8     h = act(z[:, :n]) * z[:, n:], z as in linear8 without a bias
  experts    rows offsets[g] ... offsets[g + 1] of x meet w[g]: out = act(x w[g]^T + bias[g]), or gated as above; a training
             step keeps z too
  experts_back  from dout and z: the gradients of x, and of w and bias by expert

Rows after the last offset belong to no expert; the outputs keep there what they held (zeros here). With `own` false, `run`
takes elementary torch operations in float32 and rounds once at the end; with `own` true it calls the library's kernels.
`exact` is the definition in float64.
"""

import math

import torch

own = False

DEVICE = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # one token's decoded float32 sum, before a layer in 8 bits: the call is all latency
        {"name": "quantize-token", "op": "quantize", "rows": 1, "cols": 5120, "dtype": "f32", "pad": 0},
        # a prompt's activations, the flashcomm workload's tensor: memory bounds it
        {"name": "quantize-prompt", "op": "quantize", "rows": 8192, "cols": 8192, "dtype": "bf16", "pad": 0},
        # one token through a whole layer of width 4096: the weight's bytes bound it, half of bf16's
        {"name": "int8-token", "op": "linear8", "m": 1, "n": 4096, "k": 4096, "act": "gelu", "bias": True,
         "residual": False, "out": "bf16", "pad": 0},
        # an odd-sized projection on a ragged batch: every edge inside a tile, rows that start anywhere, float32 sums
        {"name": "int8-odd", "op": "linear8", "m": 301, "n": 1001, "k": 1285, "act": "none", "bias": True,
         "residual": False, "out": "f32", "pad": 3},
        # a prompt through the flashcomm workload's layer, onto the residual stream: the matrix cores bound it
        {"name": "int8-prompt", "op": "linear8", "m": 8192, "n": 8192, "k": 8192, "act": "none", "bias": True,
         "residual": True, "out": "bf16", "pad": 0},
        # a serving batch, one token each, through one rank's share of the gated layer
        {"name": "int8-gated-batch", "op": "gated8", "m": 24, "n": 1728, "k": 5120, "act": "silu", "out": "bf16",
         "pad": 0},
        # a prompt through the gated layer at the equarx workload's width
        {"name": "int8-gated-prompt", "op": "gated8", "m": 4096, "n": 5120, "k": 5120, "act": "silu", "out": "bf16",
         "pad": 0},
        # one token that goes to eight of 64 experts: their weights' bytes bound it
        {"name": "experts-token", "op": "experts", "groups": 64, "tokens": 1, "top": 8, "spare": 0, "n": 1024, "k": 2048,
         "gated": True, "act": "silu", "bias": False, "save": False, "out": "bf16", "pad": 0},
        # a ragged batch in a buffer with room for more rows, odd sizes, rows that start anywhere
        {"name": "experts-odd", "op": "experts", "groups": 12, "tokens": 231, "top": 3, "spare": 60, "n": 777, "k": 1285,
         "gated": False, "act": "gelu", "bias": True, "save": True, "out": "bf16", "pad": 3},
        # a training step's tokens, two experts each of eight, as wide as the gpt-tp workload
        {"name": "experts-train", "op": "experts", "groups": 8, "tokens": 4096, "top": 2, "spare": 0, "n": 4096, "k": 4096,
         "gated": True, "act": "silu", "bias": False, "save": True, "out": "bf16", "pad": 0},
        # the backward pass of short sequences through many small experts with biases
        {"name": "experts-back-short", "op": "experts_back", "groups": 32, "tokens": 500, "top": 4, "spare": 48, "n": 520,
         "k": 1000, "gated": False, "act": "gelu", "bias": True, "pad": 0},
        # the backward pass of the training step
        {"name": "experts-back-train", "op": "experts_back", "groups": 8, "tokens": 4096, "top": 2, "spare": 0, "n": 4096,
         "k": 4096, "gated": True, "act": "silu", "bias": False, "pad": 0},
    ]


def _spread(rng, low, high):
    """A whole number in [low, high], even over its logarithm; one in three is odd, the others multiples of 8."""
    v = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    v = v | 1 if rng.random() < 1 / 3 else (v + 7) // 8 * 8
    return min(max(v, low), high)


MOST_PRODUCTS = 8192 ** 3          # of the largest listed cases
MOST_WEIGHTS = 8 * 8192 * 4096     # elements of all experts' weights
MOST_BYTES = 1300 << 20            # read and written at most


def draw(rng):
    op = rng.choice(["quantize", "linear8", "linear8", "gated8", "experts", "experts", "experts_back", "experts_back"])
    pad = rng.choice([0, 0, 16, 3])
    if op == "quantize":
        cols, dtype = _spread(rng, 64, 16384), rng.choice(["bf16", "bf16", "f32"])
        rows = _spread(rng, 1, 8192 * 8192 * 2 // (cols * DTYPES[dtype].itemsize))
        return {"op": op, "rows": rows, "cols": cols, "dtype": dtype, "pad": pad}
    n, k = _spread(rng, 256, 8192), _spread(rng, 256, 8192)
    if op in ("linear8", "gated8"):
        most = MOST_PRODUCTS // ((2 if op == "gated8" else 1) * n * k)
        m = 1 if rng.random() < 0.15 else _spread(rng, 2, max(2, min(16384, most)))
        case = {"op": op, "m": m, "n": n, "k": k, "out": rng.choice(["bf16", "f32"]), "pad": pad}
        if op == "linear8":
            case.update(act=rng.choice(["none", "gelu", "silu", "relu"]), bias=rng.random() < 0.7,
                        residual=rng.random() < 0.5)
        else:
            case.update(act=rng.choice(["silu", "gelu"]))
        return case
    gated = rng.random() < 0.5
    wide = 2 * n if gated else n
    while wide * k > MOST_WEIGHTS // 2:
        n, k = max(256, n // 2), max(256, k // 2)
        wide = 2 * n if gated else n
    groups = max(2, min(_spread(rng, 2, 128), MOST_WEIGHTS // (wide * k)))
    top = rng.randint(1, min(8, groups))
    most = MOST_PRODUCTS // ((2 if op == "experts_back" else 1) * wide * k * top)
    tokens = 1 if op == "experts" and rng.random() < 0.15 else _spread(rng, 2, max(2, min(8192, most)))
    case = {"op": op, "groups": groups, "tokens": tokens, "top": top, "spare": rng.choice([0, 0, rng.randint(1, 100)]),
            "n": n, "k": k, "gated": gated, "act": rng.choice(["silu", "gelu"] if gated else ["none", "gelu", "silu", "relu"]),
            "bias": not gated and rng.random() < 0.6, "pad": pad}
    if op == "experts":
        case.update(save=rng.random() < 0.4, out=rng.choice(["bf16", "f32"]))
    while work(case)["bytes"] > MOST_BYTES:
        case["tokens"] //= 2
    return case


# ----------------------------------------------------------------- inputs --

def _matrix(gen, rows, cols, sigma, dtype=torch.bfloat16, pad=0, outliers=False, mean=0.0):
    """Normal values; `outliers`: one channel in a hundred ten times as large, as hidden states have them;
    `pad`: the rows lie that many elements apart, as in a slice of a wider tensor."""
    v = torch.randn(rows, cols, generator=gen, device=DEVICE) * sigma + mean
    if outliers:
        v[:, torch.randint(0, cols, (max(1, cols // 100),), generator=gen, device=DEVICE)] *= 10.0
    wide = torch.empty(rows, cols + pad, dtype=dtype, device=DEVICE)
    wide[:, :cols] = v
    return wide[:, :cols]


def _codes(gen, rows, cols, sigma, pad, outliers):
    """8-bit codes of normal values and their scales by row."""
    v = _matrix(gen, rows, cols, sigma, torch.float32, 0, outliers)
    scale = v.abs().amax(1) / 127
    wide = torch.zeros(rows, cols + pad, dtype=torch.int8, device=DEVICE)
    wide[:, :cols] = torch.round(v / scale[:, None])
    return wide[:, :cols], scale


def _offsets(gen, tokens, top, groups):
    """Each token goes to `top` different experts, some of them far more often taken than others."""
    liked = 0.7 * torch.randn(groups, generator=gen, device=DEVICE)
    noise = torch.rand(tokens, groups, generator=gen, device=DEVICE).clamp(1e-6, 1 - 1e-6)
    taken = (liked - torch.log(-torch.log(noise))).topk(top, 1).indices
    offsets = torch.zeros(groups + 1, dtype=torch.int32, device=DEVICE)
    offsets[1:] = torch.bincount(taken.flatten(), minlength=groups).cumsum(0)
    return offsets


def _inputs(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(int(seed))
    op, pad = case["op"], case["pad"]
    if op == "quantize":
        return {"x": _matrix(gen, case["rows"], case["cols"], 1.0, DTYPES[case["dtype"]], pad, outliers=True)}
    n, k = case["n"], case["k"]
    d = {}
    if op in ("linear8", "gated8"):
        m = case["m"]
        d["x"], d["xs"] = _codes(gen, m, k, 1.0, pad, True)
        d["w"], d["ws"] = _codes(gen, 2 * n if op == "gated8" else n, k, 0.02, pad, False)
        if op == "linear8":
            d["bias"] = _matrix(gen, 1, n, 0.1)[0] if case["bias"] else None
            d["residual"] = _matrix(gen, m, n, 1.0, pad=pad) if case["residual"] else None
        return d
    groups, m = case["groups"], case["tokens"] * case["top"] + case["spare"]
    wide = 2 * n if case["gated"] else n
    d["offsets"] = _offsets(gen, case["tokens"], case["top"], groups)
    d["x"] = _matrix(gen, m, k, 1.0, pad=pad, outliers=op == "experts")
    w = _matrix(gen, groups * wide, k, 0.02, pad=pad)
    d["w"] = torch.as_strided(w, (groups, wide, k), (wide * (k + pad), k + pad, 1))
    if op == "experts":
        d["bias"] = _matrix(gen, groups, n, 0.1) if case["bias"] else None
    else:
        d["dout"] = _matrix(gen, m, n, 1e-2, pad=pad)
        # z as the forward pass keeps it: k products of x and w
        d["z"] = None if case["act"] == "none" else _matrix(gen, m, wide, 0.02 * math.sqrt(k), pad=pad)
    return d


def prepare(case, seed):
    """Inputs, and the outputs' buffers that a program which calls the library again and again keeps (zeros: rows of no
    expert stay what they were)."""
    s = dict(_inputs(case, seed), case=dict(case))

    def new(dtype, *shape):
        return torch.zeros(*shape, dtype=dtype, device=DEVICE)

    op, bf16, f32 = case["op"], torch.bfloat16, torch.float32
    if op == "quantize":
        s.update(q=new(torch.int8, case["rows"], case["cols"]), scale=new(f32, case["rows"]))
    elif op in ("linear8", "gated8"):
        s["out"] = new(DTYPES[case["out"]], case["m"], case["n"])
    else:
        groups, m = case["groups"], s["x"].shape[0]
        n, k = case["n"], case["k"]
        wide = 2 * n if case["gated"] else n
        if op == "experts":
            s["out"] = new(DTYPES[case["out"]], m, n)
            s["keep"] = new(bf16, m, wide) if case["save"] else None
        else:
            s["dx"], s["dw"] = new(bf16, m, k), new(bf16, groups, wide, k)
            s["dbias"] = new(f32, groups, n) if case["bias"] else None
    return s


# -------------------------------------------------------------- plain form --

def _act(z, act):
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    return z


def _act_slope(z, act):
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return s * (1.0 + z * (1.0 - s))
    if act == "relu":
        return (z > 0).to(z.dtype)
    return torch.ones_like(z)


def _ranges(s):
    o = s["offsets"].tolist()
    return list(enumerate(zip(o, o[1:])))


def _whole(parts, m):
    """The experts' rows one after the other, then zeros: the rows of no expert."""
    v = torch.cat(parts)
    return torch.cat([v, v.new_zeros(m - v.shape[0], v.shape[1])])


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op == "quantize":
        x = s["x"].float()
        largest = x.abs().amax(1)
        zero = largest < 2.0 ** -100
        scale = torch.where(zero, torch.zeros_like(largest), largest / 127.0)
        inv = torch.where(zero, torch.zeros_like(largest), 127.0 / largest)
        return {"codes": torch.round(x * inv[:, None]).to(torch.int8), "scale": scale}
    if op in ("linear8", "gated8"):
        z = (s["x"].float() @ s["w"].float().t()) * s["xs"][:, None] * s["ws"]
        if op == "gated8":
            n = c["n"]
            return {"out": (_act(z[:, :n], c["act"]) * z[:, n:]).to(DTYPES[c["out"]])}
        if s["bias"] is not None:
            z = z + s["bias"].float()
        out = _act(z, c["act"])
        if s["residual"] is not None:
            out = out + s["residual"].float()
        return {"out": out.to(DTYPES[c["out"]])}
    m, n, w = s["x"].shape[0], c["n"], s["w"]
    if op == "experts":
        x = s["x"].float()
        z = _whole([x[a:b] @ w[g].float().t() + (0.0 if s["bias"] is None else s["bias"][g].float())
                    for g, (a, b) in _ranges(s)], m)
        out = _act(z[:, :n], c["act"]) * z[:, n:] if c["gated"] else _act(z, c["act"])
        r = {"out": out.to(DTYPES[c["out"]])}
        if c["save"]:
            r["z"] = z.to(torch.bfloat16)
        return r
    dout, x = s["dout"].float(), s["x"].float()
    if c["gated"]:
        z = s["z"].float()
        gate, up = z[:, :n], z[:, n:]
        dz = torch.cat([dout * up * _act_slope(gate, c["act"]), dout * _act(gate, c["act"])], 1)
    else:
        dz = dout if c["act"] == "none" else dout * _act_slope(s["z"].float(), c["act"])
    r = {"dx": _whole([dz[a:b] @ w[g].float() for g, (a, b) in _ranges(s)], m).to(torch.bfloat16),
         "dw": torch.stack([dz[a:b].t() @ x[a:b] for g, (a, b) in _ranges(s)]).to(torch.bfloat16)}
    if c["bias"]:
        r["dbias"] = torch.stack([dz[a:b].sum(0) for g, (a, b) in _ranges(s)])
    return r


# ------------------------------------------------------------ the library --

def _workspace(s, name, *sizes):
    """The call's workspace, which the program keeps from its first call on."""
    if "workspace" not in s:
        import quantized_compression_tensor_amd as T
        size = getattr(T, name + "_workspace_bytes")(*sizes)
        s["workspace"] = torch.empty(size, dtype=torch.uint8, device=DEVICE) if size else None
    return s["workspace"]


def _library(s):
    import quantized_compression_tensor_amd as T
    c = s["case"]
    op = c["op"]
    if op == "quantize":
        T.taco_quantize_rows(s["x"], s["q"], s["scale"])
        return {"codes": s["q"], "scale": s["scale"]}
    act = {"none": T.TACO_ACT_NONE, "gelu": T.TACO_ACT_GELU, "silu": T.TACO_ACT_SILU, "relu": T.TACO_ACT_RELU}[c["act"]]
    n, k = c["n"], c["k"]
    if op == "linear8":
        T.taco_linear_int8(s["x"], s["xs"], s["w"], s["ws"], s["out"], bias=s["bias"], act=act, residual=s["residual"],
                           workspace=_workspace(s, "taco_linear_int8", c["m"], n, k))
        return {"out": s["out"]}
    if op == "gated8":
        T.taco_gated_linear_int8(s["x"], s["xs"], s["w"], s["ws"], s["out"], act=act,
                                 workspace=_workspace(s, "taco_gated_linear_int8", c["m"], n, k))
        return {"out": s["out"]}
    sizes = (c["groups"], s["x"].shape[0], n, k)
    if op == "experts":
        if c["gated"]:
            T.taco_grouped_gated_linear(s["x"], s["w"], s["offsets"], s["out"], act=act, preact=s["keep"],
                                        workspace=_workspace(s, "taco_grouped_gated_linear", *sizes))
        else:
            T.taco_grouped_linear(s["x"], s["w"], s["offsets"], s["out"], bias=s["bias"], act=act, preact=s["keep"],
                                  workspace=_workspace(s, "taco_grouped_linear", *sizes))
        return {"out": s["out"], "z": s["keep"]} if c["save"] else {"out": s["out"]}
    if c["gated"]:
        T.taco_grouped_gated_linear_backward(s["dout"], s["x"], s["w"], s["offsets"], act=act, preact=s["z"], dx=s["dx"],
                                             dw=s["dw"],
                                             workspace=_workspace(s, "taco_grouped_gated_linear_backward", *sizes))
    else:
        T.taco_grouped_linear_backward(s["dout"], s["x"], s["w"], s["offsets"], act=act, preact=s["z"], dx=s["dx"],
                                       dw=s["dw"], dbias=s["dbias"],
                                       workspace=_workspace(s, "taco_grouped_linear_backward", *sizes))
    r = {"dx": s["dx"], "dw": s["dw"]}
    if c["bias"]:
        r["dbias"] = s["dbias"]
    return r


def run(state):
    return _library(state) if own else _plain(state)


# ------------------------------------------------------ sizes and the truth --

def work(case):
    op = case["op"]
    if op == "quantize":
        rows, cols = case["rows"], case["cols"]
        return {"bytes": rows * cols * (DTYPES[case["dtype"]].itemsize + 1) + 4 * rows, "flops": 3 * rows * cols}
    n, k = case["n"], case["k"]
    if op in ("linear8", "gated8"):
        m, wide = case["m"], 2 * n if op == "gated8" else n
        size = m * k + wide * k + 4 * (m + wide) + m * n * DTYPES[case["out"]].itemsize
        if op == "linear8":
            size += (2 * n if case["bias"] else 0) + (2 * m * n if case["residual"] else 0)
        return {"bytes": size, "flops": 2 * m * wide * k}
    rows, wide, groups = case["tokens"] * case["top"], 2 * n if case["gated"] else n, case["groups"]
    read = 2 * rows * k + 2 * min(groups, rows) * wide * k + 4 * groups     # at most so many experts have a row
    if op == "experts":
        size = read + rows * n * DTYPES[case["out"]].itemsize + (2 * rows * wide if case["save"] else 0)
        return {"bytes": size + (2 * min(groups, rows) * n if case["bias"] else 0), "flops": 2 * rows * wide * k}
    size = read + 2 * rows * n + 2 * rows * k + 2 * groups * wide * k
    if case["act"] != "none":
        size += 2 * rows * wide
    return {"bytes": size + (4 * groups * n if case["bias"] else 0), "flops": 4 * rows * wide * k}


def exact(case, seed):
    """The definitions, in float64."""
    d = _inputs(case, seed)
    op = case["op"]
    if op == "quantize":
        # a code is a rounding to whole numbers in float32's steps: no value of its own in 64 bits
        return {"codes": None, "scale": torch.linalg.vector_norm(d["x"].double(), math.inf, 1) / 127}

    def phi(t):      # the normal distribution's function: gelu(t) = t phi(t), its slope phi(t) + t phi'(t)
        return torch.special.ndtr(t)

    def value(t):
        return {"none": lambda: t, "relu": lambda: t.clamp(min=0), "silu": lambda: t * torch.sigmoid(t),
                "gelu": lambda: t * phi(t)}[case["act"]]()

    def slope(t):
        return {"none": lambda: torch.ones_like(t), "relu": lambda: (t > 0).double(),
                "silu": lambda: torch.sigmoid(t) + t * torch.sigmoid(t) * torch.sigmoid(-t),
                "gelu": lambda: phi(t) + t * torch.exp(-t.square() / 2) / math.sqrt(2 * math.pi)}[case["act"]]()

    n = case["n"]
    if op in ("linear8", "gated8"):
        z = torch.mm(d["x"].double() * d["xs"].double()[:, None], (d["w"].double() * d["ws"].double()[:, None]).t())
        if op == "gated8":
            return {"out": value(z[:, :n]).mul_(z[:, n:])}
        z = z if d["bias"] is None else z.add_(d["bias"].double())
        out = value(z)
        return {"out": out if d["residual"] is None else out + d["residual"].double()}
    x, o = d["x"].double(), d["offsets"].cpu()
    m, k, groups = x.shape[0], case["k"], case["groups"]
    wide = d["w"].shape[1]

    def zeros(*shape):
        return torch.zeros(*shape, dtype=torch.float64, device=DEVICE)

    if op == "experts":
        z, out = zeros(m, wide), zeros(m, n)
        for g in range(groups):
            r = slice(int(o[g]), int(o[g + 1]))
            z[r] = torch.mm(x[r], d["w"][g].double().t())
            if d["bias"] is not None:
                z[r] += d["bias"][g].double()
            out[r] = value(z[r, :n]) * z[r, n:] if case["gated"] else value(z[r])
        return {"out": out, "z": z} if case["save"] else {"out": out}
    dx, dw, db = zeros(m, k), zeros(groups, wide, k), zeros(groups, n)
    for g in range(groups):
        r = slice(int(o[g]), int(o[g + 1]))
        dz = d["dout"][r].double()
        if case["gated"]:
            t, u = d["z"][r, :n].double(), d["z"][r, n:].double()
            dz = torch.cat([dz * u * slope(t), dz * value(t)], 1)
        elif case["act"] != "none":
            dz = dz * slope(d["z"][r].double())
        dx[r] = torch.mm(dz, d["w"][g].double())
        dw[g] = torch.mm(dz.t(), x[r])
        if case["bias"]:
            db[g] = dz.sum(0)
    return {"dx": dx, "dw": dw, "dbias": db} if case["bias"] else {"dx": dx, "dw": dw}
