"""The operators of a feed-forward sub-layer, as cases to be timed and compared.

A tensor-parallel feed-forward sub-layer is a layer norm, one or two projections with an activation, and a projection
back, whose partial sums the codecs of this library compress; in training each has its backward pass. A case is one
operator in one direction at one size:

  norm       y = (x - mean) * rstd * weight + bias, by row, with mean and rstd kept for the backward pass
  norm_back  the gradients of x, weight and bias
  linear     out = act(x w^T + bias) + residual; a training step keeps z = x w^T + bias too
  linear_back  from dout and z: the gradients of x, w and bias
  gated      h = act(x wg^T) * (x wu^T), w = [wg; wu]; a training step keeps z = x w^T too
  gated_back   from dh and z: the gradients of x and w

With `own` false, `run` takes elementary torch operations in float32 and rounds once at the end; with `own` true it
calls the library's kernels. `exact` is the definition in float64.
"""

import math

import torch

own = False

EPS = 1e-5
DEVICE = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # one token of a serving step: the call is all latency
        {"name": "norm-token", "op": "norm", "rows": 1, "cols": 4096, "dtype": "bf16", "pad": 0},
        # a prompt's activations, as wide as the equarx workload's
        {"name": "norm-prompt", "op": "norm", "rows": 8192, "cols": 5120, "dtype": "bf16", "pad": 0},
        # a short ragged batch of decoded float32 sums, odd width: rows start at 4-byte boundaries
        {"name": "norm-back-odd", "op": "norm_back", "rows": 777, "cols": 1025, "dtype": "f32", "pad": 0},
        # the qwen-tp workload's tensor in a training step
        {"name": "norm-back-train", "op": "norm_back", "rows": 32768, "cols": 5120, "dtype": "bf16", "pad": 0},
        # one token through a whole layer of width 4096: the weight's bytes bound it
        {"name": "linear-token", "op": "linear", "m": 1, "n": 4096, "k": 4096, "act": "gelu", "bias": True,
         "residual": False, "save": False, "out": "bf16", "pad": 0},
        # a prompt through the flashcomm workload's layer, onto the residual stream: the matrix cores bound it
        {"name": "linear-prompt", "op": "linear", "m": 8192, "n": 8192, "k": 8192, "act": "none", "bias": True,
         "residual": True, "save": False, "out": "bf16", "pad": 0},
        # an odd-sized projection on a ragged batch: every edge inside a tile, rows at 2-byte boundaries
        {"name": "linear-back-odd", "op": "linear_back", "m": 1001, "n": 777, "k": 1285, "act": "gelu", "bias": True,
         "grad": "bf16", "pad": 3},
        # the gpt-tp workload's tensor and layer in a training step
        {"name": "linear-back-train", "op": "linear_back", "m": 4096, "n": 4096, "k": 4096, "act": "gelu",
         "bias": True, "grad": "bf16", "pad": 0},
        # a serving batch, one token each, through one rank's share of the gated layer
        {"name": "gated-batch", "op": "gated", "m": 24, "n": 1728, "k": 5120, "act": "silu", "save": False,
         "out": "bf16", "pad": 0},
        # a training step's forward pass of it, the projections kept
        {"name": "gated-train", "op": "gated", "m": 4096, "n": 5120, "k": 5120, "act": "silu", "save": True,
         "out": "bf16", "pad": 0},
        # a small model's layer on one short sequence: fewer tiles than compute units
        {"name": "gated-back-short", "op": "gated_back", "m": 512, "n": 1400, "k": 1024, "act": "silu",
         "grad": "bf16", "pad": 0},
        # the backward pass at the equarx workload's sizes
        {"name": "gated-back-train", "op": "gated_back", "m": 8192, "n": 5120, "k": 5120, "act": "silu",
         "grad": "bf16", "pad": 0},
    ]


def _spread(rng, low, high):
    """A whole number in [low, high], even over its logarithm; one in three is odd, the others multiples of 8."""
    v = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    v = v | 1 if rng.random() < 1 / 3 else (v + 7) // 8 * 8
    v += 8 if v == 3072 else 0     # a usual size elsewhere, none of this library's
    return min(max(v, low), high)


def draw(rng):
    op = rng.choice(["norm", "norm_back", "linear", "linear_back", "gated", "gated_back"])
    pad = rng.choice([0, 0, 8, 3])
    if op in ("norm", "norm_back"):
        cols = _spread(rng, 128, 8192)
        dtype = rng.choice(["bf16", "bf16", "f32"])
        rows = _spread(rng, 1, 32768 * 5120 * 2 // (max(cols, 5120) * DTYPES[dtype].itemsize))
        return {"op": op, "rows": rows, "cols": cols, "dtype": dtype, "pad": pad}
    n, k = _spread(rng, 256, 8192), _spread(rng, 256, 8192)
    # at most the largest listed case's products
    products = {"linear": 1, "linear_back": 2, "gated": 2, "gated_back": 4}[op]
    most = 4 * 8192 * 5120 * 5120 // (products * n * k)
    m = 1 if rng.random() < 0.15 else _spread(rng, 2, max(2, min(8192, most)))
    case = {"op": op, "m": m, "n": n, "k": k, "pad": pad}
    if op == "linear":
        case.update(act=rng.choice(["none", "gelu", "silu", "relu"]), bias=rng.random() < 0.7,
                    residual=rng.random() < 0.5, save=rng.random() < 0.3, out=rng.choice(["bf16", "f32"]))
    elif op == "linear_back":
        # gradients in float32 where no activation lies between them and their inputs
        act = rng.choice(["none", "gelu", "silu", "relu"])
        case.update(act=act, bias=rng.random() < 0.7, grad=rng.choice(["bf16", "f32"]) if act == "none" else "bf16")
    elif op == "gated":
        case.update(act=rng.choice(["silu", "gelu"]), save=rng.random() < 0.5, out=rng.choice(["bf16", "f32"]))
    else:
        case.update(act=rng.choice(["silu", "gelu"]), grad="bf16")
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


def _inputs(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(int(seed))
    op, pad = case["op"], case["pad"]
    if op in ("norm", "norm_back"):
        rows, cols, dt = case["rows"], case["cols"], DTYPES[case["dtype"]]
        x = _matrix(gen, rows, cols, 1.0, dt, pad, outliers=True, mean=0.1)
        d = {"x": x, "weight": _matrix(gen, 1, cols, 0.1, dt, mean=1.0)[0], "bias": _matrix(gen, 1, cols, 0.1, dt)[0]}
        if op == "norm_back":
            d["dy"] = _matrix(gen, rows, cols, 1e-2, dt, pad)
            # what a forward pass has kept
            d["mean"] = x.float().mean(1)
            d["rstd"] = (x.float().var(1, unbiased=False) + EPS).rsqrt()
        return d
    m, n, k = case["m"], case["n"], case["k"]
    wide = 2 * n if op.startswith("gated") else n
    d = {"x": _matrix(gen, m, k, 1.0, pad=pad, outliers=op in ("linear", "gated"))}
    d["w"] = _matrix(gen, wide, k, 0.02, pad=pad)
    if op == "linear":
        d["bias"] = _matrix(gen, 1, n, 0.1)[0] if case["bias"] else None
        d["residual"] = _matrix(gen, m, n, 1.0, pad=pad) if case["residual"] else None
    elif op in ("linear_back", "gated_back"):
        d["dout"] = _matrix(gen, m, n, 1e-2, pad=pad)
        # z as the forward pass keeps it: k products of x and w
        d["z"] = None if case["act"] == "none" else _matrix(gen, m, wide, 0.02 * math.sqrt(k), pad=pad)
    return d


def prepare(case, seed):
    """Inputs, and the buffers that a program which calls the library again and again keeps: outputs and workspace."""
    s = dict(_inputs(case, seed), case=dict(case))

    def new(dtype, *shape):
        return torch.empty(*shape, dtype=dtype, device=DEVICE)

    op = case["op"]
    if op == "norm":
        rows, cols, dt = case["rows"], case["cols"], DTYPES[case["dtype"]]
        s.update(y=new(dt, rows, cols), mean=new(torch.float32, rows), rstd=new(torch.float32, rows))
    elif op == "norm_back":
        rows, cols, dt = case["rows"], case["cols"], DTYPES[case["dtype"]]
        s.update(dx=new(dt, rows, cols), dweight=new(torch.float32, cols), dbias=new(torch.float32, cols))
    elif op in ("linear", "gated"):
        m, n = case["m"], case["n"]
        s["out"] = new(DTYPES[case["out"]], m, n)
        s["keep"] = new(torch.bfloat16, m, 2 * n if op == "gated" else n) if case["save"] else None
    else:
        m, n, k = case["m"], case["n"], case["k"]
        s["dx"] = new(torch.bfloat16, m, k)
        s["dw"] = new(DTYPES[case["grad"]], 2 * n if op == "gated_back" else n, k)
        s["dbias"] = new(torch.float32, n) if op == "linear_back" and case["bias"] else None
    if own:
        import quantized_compression_tensor_amd as T
        if op == "norm_back":
            size = T.taco_layer_norm_backward_workspace_bytes(case["rows"], case["cols"])
        elif op == "norm":
            size = 0
        else:
            size = getattr(T, {"linear": "taco_linear_workspace_bytes", "linear_back": "taco_linear_backward_workspace_bytes",
                               "gated": "taco_gated_linear_workspace_bytes",
                               "gated_back": "taco_gated_linear_backward_workspace_bytes"}[op])(case["m"], case["n"], case["k"])
        s["workspace"] = new(torch.uint8, size) if size else None
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


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op == "norm":
        x = s["x"].float()
        mean = x.mean(1)
        d = x - mean[:, None]
        rstd = 1.0 / torch.sqrt((d * d).mean(1) + EPS)
        y = d * rstd[:, None] * s["weight"].float() + s["bias"].float()
        return {"y": y.to(s["x"].dtype), "mean": mean, "rstd": rstd}
    if op == "norm_back":
        dy = s["dy"].float()
        xhat = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
        g = dy * s["weight"].float()
        dx = (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True)) * s["rstd"][:, None]
        return {"dx": dx.to(s["x"].dtype), "dweight": (dy * xhat).sum(0), "dbias": dy.sum(0)}
    x, w = s["x"].float(), s["w"].float()
    if op == "linear":
        z = x @ w.t()
        if s["bias"] is not None:
            z = z + s["bias"].float()
        out = _act(z, c["act"])
        if s["residual"] is not None:
            out = out + s["residual"].float()
        r = {"out": out.to(DTYPES[c["out"]])}
        if c["save"]:
            r["z"] = z.to(torch.bfloat16)
        return r
    if op == "gated":
        z = x @ w.t()
        n = c["n"]
        r = {"out": (_act(z[:, :n], c["act"]) * z[:, n:]).to(DTYPES[c["out"]])}
        if c["save"]:
            r["z"] = z.to(torch.bfloat16)
        return r
    dout = s["dout"].float()
    if op == "linear_back":
        dz = dout if c["act"] == "none" else dout * _act_slope(s["z"].float(), c["act"])
        r = {"dx": (dz @ w).to(torch.bfloat16), "dw": (dz.t() @ x).to(DTYPES[c["grad"]])}
        if c["bias"]:
            r["dbias"] = dz.sum(0)
        return r
    z, n = s["z"].float(), c["n"]
    gate, up = z[:, :n], z[:, n:]
    dz = torch.cat([dout * up * _act_slope(gate, c["act"]), dout * _act(gate, c["act"])], 1)
    return {"dx": (dz @ w).to(torch.bfloat16), "dw": (dz.t() @ x).to(DTYPES[c["grad"]])}


# ------------------------------------------------------------ the library --

def _library(s):
    import quantized_compression_tensor_amd as T
    c = s["case"]
    op = c["op"]
    if op == "norm":
        T.taco_layer_norm(s["x"], s["weight"], s["bias"], EPS, s["y"], mean=s["mean"], rstd=s["rstd"])
        return {"y": s["y"], "mean": s["mean"], "rstd": s["rstd"]}
    if op == "norm_back":
        T.taco_layer_norm_backward(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"], dx=s["dx"],
                                   dweight=s["dweight"], dbias=s["dbias"], workspace=s["workspace"])
        return {"dx": s["dx"], "dweight": s["dweight"], "dbias": s["dbias"]}
    act = {"none": T.TACO_ACT_NONE, "gelu": T.TACO_ACT_GELU, "silu": T.TACO_ACT_SILU, "relu": T.TACO_ACT_RELU}[c["act"]]
    if op == "linear":
        T.taco_linear(s["x"], s["w"], s["out"], bias=s["bias"], act=act, residual=s["residual"], preact=s["keep"],
                      workspace=s["workspace"])
    elif op == "gated":
        T.taco_gated_linear(s["x"], s["w"], s["out"], act=act, preact=s["keep"], workspace=s["workspace"])
    if op in ("linear", "gated"):
        return {"out": s["out"], "z": s["keep"]} if c["save"] else {"out": s["out"]}
    if op == "linear_back":
        T.taco_linear_backward(s["dout"], s["x"], s["w"], act=act, preact=s["z"], dx=s["dx"], dw=s["dw"],
                               dbias=s["dbias"], workspace=s["workspace"])
        r = {"dx": s["dx"], "dw": s["dw"]}
        if c["bias"]:
            r["dbias"] = s["dbias"]
        return r
    T.taco_gated_linear_backward(s["dout"], s["x"], s["w"], act=act, preact=s["z"], dx=s["dx"], dw=s["dw"],
                                 workspace=s["workspace"])
    return {"dx": s["dx"], "dw": s["dw"]}


def run(state):
    return _library(state) if own else _plain(state)


# ------------------------------------------------------ sizes and the truth --

def work(case):
    op = case["op"]
    if op in ("norm", "norm_back"):
        rows, cols, b = case["rows"], case["cols"], DTYPES[case["dtype"]].itemsize
        if op == "norm":
            return {"bytes": 2 * rows * cols * b + 2 * cols * b + 8 * rows, "flops": 8 * rows * cols}
        return {"bytes": 3 * rows * cols * b + cols * b + 8 * rows + 8 * cols, "flops": 14 * rows * cols}
    m, n, k = case["m"], case["n"], case["k"]
    wide = 2 * n if op.startswith("gated") else n
    read = 2 * (m * k + wide * k)
    if op in ("linear", "gated"):
        size = read + m * n * DTYPES[case["out"]].itemsize + (2 * m * wide if case["save"] else 0)
        if op == "linear":
            size += (2 * n if case["bias"] else 0) + (2 * m * n if case["residual"] else 0)
        return {"bytes": size, "flops": 2 * m * wide * k}
    size = read + 2 * m * n + 2 * m * k + wide * k * DTYPES[case["grad"]].itemsize
    if case["act"] != "none":
        size += 2 * m * wide
    if op == "linear_back" and case["bias"]:
        size += 4 * n
    return {"bytes": size, "flops": 4 * m * wide * k}


def exact(case, seed):
    """The definitions, in float64."""
    d = {k: v if v is None else v.double() for k, v in _inputs(case, seed).items()}
    op = case["op"]
    half = torch.tensor(0.5, dtype=torch.float64, device=DEVICE)

    def phi(t):      # the normal distribution's function: gelu(t) = t phi(t), its slope phi(t) + t phi'(t)
        return torch.special.ndtr(t)

    def value(t, act):
        return {"none": lambda: t, "relu": lambda: t.clamp(min=0), "silu": lambda: t * torch.sigmoid(t),
                "gelu": lambda: t * phi(t)}[act]()

    def slope(t, act):
        return {"none": lambda: torch.ones_like(t), "relu": lambda: torch.heaviside(t, 0 * half),
                "silu": lambda: torch.sigmoid(t) + t * torch.sigmoid(t) * torch.sigmoid(-t),
                "gelu": lambda: phi(t) + t * torch.exp(-half * t.square()) * (half / math.pi).sqrt()}[act]()

    if op == "norm":
        var, mean = torch.var_mean(d["x"], 1, correction=0)
        rstd = (var + EPS).rsqrt()
        return {"y": torch.addcmul(d["bias"], (d["x"] - mean[:, None]).mul(rstd[:, None]), d["weight"]),
                "mean": mean, "rstd": rstd}
    if op == "norm_back":
        # the Jacobian of row r: rstd (I - 1 1^T / cols - xhat xhat^T / cols) diag(weight)
        cols = case["cols"]
        xhat = d["x"].sub(d["mean"][:, None]).mul(d["rstd"][:, None])
        g = d["dy"] * d["weight"]
        along = torch.stack([g.sum(1), (g * xhat).sum(1)], 1) / cols
        dx = (g - along[:, :1] - xhat * along[:, 1:]) * d["rstd"][:, None]
        return {"dx": dx, "dweight": (d["dy"] * xhat).sum(0), "dbias": d["dy"].sum(0)}
    n = case["n"]
    if op == "linear":
        z = torch.mm(d["x"], d["w"].t())
        z = z if d["bias"] is None else z + d["bias"]
        out = value(z, case["act"])
        out = out if d["residual"] is None else out + d["residual"]
        return {"out": out, "z": z} if case["save"] else {"out": out}
    if op == "gated":
        gate, up = torch.mm(d["x"], d["w"][:n].t()), torch.mm(d["x"], d["w"][n:].t())
        out = value(gate, case["act"]) * up
        return {"out": out, "z": torch.cat([gate, up], 1)} if case["save"] else {"out": out}
    if op == "linear_back":
        dz = d["dout"] if d["z"] is None else d["dout"] * slope(d["z"], case["act"])
        r = {"dx": torch.mm(dz, d["w"]), "dw": torch.mm(dz.t(), d["x"])}
        return dict(r, dbias=dz.sum(0)) if case["bias"] else r
    dgate = d["dout"] * d["z"][:, n:] * slope(d["z"][:, :n], case["act"])
    dup = d["dout"] * value(d["z"][:, :n], case["act"])
    return {"dx": torch.mm(dgate, d["w"][:n]) + torch.mm(dup, d["w"][n:]),
            "dw": torch.cat([torch.mm(dgate.t(), d["x"]), torch.mm(dup.t(), d["x"])], 0)}
