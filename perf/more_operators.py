"""What is measured of the operators on rows held in 8-bit integers.

Three operators that share one format, int8 values with a float32 scale for
each row or for each group of columns of a row: the layer norm, which writes
such rows (or e4m3 ones, or the storage type), and its backward; the matrix
product in 8-bit integers with scales for each token and channel; and
activation checkpoints, packed in the forward and read by the product's
backward. The sizes are those of the workloads the library is benchmarked on
(8192 x 8192 at r = 384, 28672 x 8192, 4096 x 4096), plus odd ones.

With ``own`` false, run() computes the plain form in fp32 with elementary
torch operations (a value beside the border of two 8-bit steps in 64 bits);
with ``own`` true it calls libdora.
"""

import math

import torch

own = False

FP = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
E4M3_MAX = 448.0
INT8_MAX = 127.0
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


def listed():
    return [
        # Prefill of 8192 tokens at the headline width, output in e4m3 for the next product.
        {"name": "layer norm prefill 8 bit", "op": "norm", "dtype": "bf16", "T": 8192, "d": 8192, "out": "e4m3"},
        # A ragged batch at a width that no vector load divides.
        {"name": "layer norm ragged f16", "op": "norm", "dtype": "f16", "T": 777, "d": 3583, "out": "same"},
        # One training step's backward of the norm, 8192 tokens of a 4096-wide model.
        {"name": "layer norm backward", "op": "norm_backward", "dtype": "bf16", "T": 8192, "d": 4096},
        # Decoding one sequence: the norm writes int8 rows, the product of integers reads them.
        {"name": "norm and product one token", "op": "norm_product", "dtype": "bf16", "T": 1, "N": 8192, "d": 8192,
         "act": "none"},
        # Decoding 16 sequences through an int8 MLP up projection with an unmerged adapter of rank 384.
        {"name": "int8 product 16 tokens", "op": "product", "dtype": "bf16", "M": 16, "N": 28672, "K": 8192, "r": 384,
         "act": "silu", "residual": False, "save": False},
        # Odd sizes in fp16: no row of x or w starts on a vector boundary.
        {"name": "int8 product ragged", "op": "product", "dtype": "f16", "M": 333, "N": 1001, "K": 777, "r": 24,
         "act": "relu", "residual": True, "save": False},
        # The whole adapted layer at the headline sizes on an int8 base: 8192 tokens, r = 384, u kept for the backward.
        {"name": "int8 product headline", "op": "product", "dtype": "bf16", "M": 8192, "N": 8192, "K": 8192, "r": 384,
         "act": "none", "residual": True, "save": True},
        # Prefill through the int8 MLP up projection.
        {"name": "int8 product prefill", "op": "product", "dtype": "bf16", "M": 8192, "N": 28672, "K": 8192, "r": 0,
         "act": "gelu_tanh", "residual": False, "save": False},
        # A layer's activations packed in the forward and restored in the backward, groups of 128 columns.
        {"name": "checkpoint round trip", "op": "checkpoint", "dtype": "bf16", "T": 8192, "d": 8192, "group": 128},
        # Training backward of a projection from packed u and x: gradients of x, W, bias and column scale.
        {"name": "checkpoint layer backward", "op": "backward", "dtype": "bf16", "M": 4096, "N": 4096, "K": 4096,
         "act": "silu", "u8": 128, "x8": 128, "w8": False, "dx": True, "dw": True},
        # The adapter's A at the headline sizes: dA = dt^T x with x packed.
        {"name": "checkpoint adapter backward", "op": "backward", "dtype": "bf16", "M": 8192, "N": 384, "K": 8192,
         "act": "none", "u8": -1, "x8": 128, "w8": False, "dx": False, "dw": True},
        # A frozen int8 base: the gradient of its input, u packed.
        {"name": "int8 base backward", "op": "backward", "dtype": "bf16", "M": 8192, "N": 8192, "K": 4096,
         "act": "gelu", "u8": 128, "x8": -1, "w8": True, "dx": True, "dw": False},
    ]


def _size(rng, low, high):
    """A size between low and high, even over its logarithm, and often odd."""
    n = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    how = rng.random()
    if how < 0.35 and n >= 128:
        n = n // 64 * 64
    elif how < 0.55 and n >= 16:
        n = n // 8 * 8
    return max(low, min(high, n))


def draw(rng):
    op = rng.choice(["norm", "norm_backward", "norm_product", "product", "product", "product", "checkpoint", "backward",
                     "backward"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "norm":
        return {"op": op, "dtype": dtype, "T": _size(rng, 1, 8192), "d": _size(rng, 256, 8192),
                "out": rng.choice(["same", "e4m3"])}
    if op == "norm_backward":
        return {"op": op, "dtype": dtype, "T": _size(rng, 1, 8192), "d": _size(rng, 256, 8192)}
    if op == "norm_product":
        # (16 bits: a sum behind 8-bit rows that the norm's last bits decide is no figure of 32)
        dtype = rng.choice(["bf16", "f16"])
        return {"op": op, "dtype": dtype, "T": _size(rng, 1, 64), "N": _size(rng, 128, 8192),
                "d": _size(rng, 256, 8192), "act": rng.choice(ACTS)}
    if op == "product":
        r = 0 if dtype == "f32" else rng.choice([0, _size(rng, 4, 768)])
        return {"op": op, "dtype": dtype, "M": _size(rng, 1, 8192), "N": _size(rng, 128, 8192),
                "K": _size(rng, 128, 8192), "r": r, "act": rng.choice(ACTS), "residual": rng.random() < 0.5,
                "save": rng.random() < 0.3}
    if op == "checkpoint":
        return {"op": op, "dtype": dtype, "T": _size(rng, 1, 8192), "d": _size(rng, 128, 8192),
                "group": rng.choice([0, 32, 64, 128, 128, 256])}
    top = 1024 if dtype == "f32" else 8192
    dx = rng.random() < 0.7
    dw = not dx or rng.random() < 0.6
    groups = [-1, 0, 64, 128]   # -1: in the storage type; 0: one scale a row
    return {"op": op, "dtype": dtype, "M": _size(rng, 16, top), "N": _size(rng, 64, top), "K": _size(rng, 128, top),
            "act": rng.choice(ACTS), "u8": rng.choice(groups), "x8": rng.choice([0, 64, 128]) if dw else -1,
            "w8": dx and (not dw or rng.random() < 0.5), "dx": dx, "dw": dw}


def _groups(v, group):
    """v [T, d] as [T, groups, columns of a group], zeros past d; group 0 is the whole row."""
    T, d = v.shape
    g = group or d
    n = -(-d // g)
    if n * g > d:
        v = torch.cat([v, v.new_zeros(T, n * g - d)], 1)
    return v.reshape(T, n, g)


def _pack(v, group):
    """Int8 rows of fp32 v: (q int8 [T, d], scale float32 [T, groups], or [T] for whole rows)."""
    T, d = v.shape
    v = _groups(v, group)
    scale = v.abs().amax(2) / INT8_MAX
    scale = torch.where(scale == 0, torch.ones_like(scale), scale)
    q = torch.round(v.double() / scale.double()[:, :, None])
    q = q.reshape(T, -1)[:, :d].to(torch.int8).contiguous()
    return q, scale if group else scale.reshape(T)


def _unpack(q, scale, group):
    """q * scale in the scale's precision."""
    T, d = q.shape
    v = _groups(q.to(scale.dtype), group) * scale.reshape(T, -1, 1)
    return v.reshape(T, -1)[:, :d]


def _rows_in_e4m3(v):
    scale = v.abs().amax(1) / E4M3_MAX
    scale = torch.where(scale == 0, torch.ones_like(scale), scale)
    return (v / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0, mean=0.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=gen, device="cuda") * std + mean).to(dtype)

    def loud(d):   # a residual stream and the activations after it have a few channels far larger than the rest
        return torch.where(torch.rand(d, generator=gen, device="cuda") < 0.003, 20.0, 1.0)

    dt = FP[case["dtype"]]
    st = {"case": case, "dt": dt, "eps": 1e-5}
    if case["op"] in ("norm", "norm_backward", "norm_product"):
        T, d = case["T"], case["d"]
        st["weight"] = normal(d, std=0.1, mean=1.0)
        # (the stream has a mean of its own, which is what the layer norm takes out)
        stream = (normal(T, d, mean=0.2) * loud(d)).to(dt)
        if case["op"] == "norm_backward":
            st["h"] = stream
            v = stream.float()
            st["mean"] = v.mean(1)
            st["rstd"] = ((v - st["mean"][:, None]).square().mean(1) + st["eps"]).rsqrt()
            st["dy"] = normal(T, d, dtype=dt)
            st["dh"] = normal(T, d, dtype=dt)
            st["dx"] = torch.empty_like(stream)
            return st
        st["norm_bias"] = normal(d, std=0.1)
        st["x"] = normal(T, d, std=0.3, dtype=dt)
        st["residual"] = stream
        st["h"] = torch.empty_like(stream)
        if case["op"] == "norm_product":
            N = case["N"]
            st["w"], st["w_scale"] = _pack(normal(N, d, std=d ** -0.5), 0)
            st["col_scale"] = normal(N, std=0.0015, mean=1.0)
            st["bias"] = normal(N, std=0.1)
            st["q"] = torch.empty(T, d, device="cuda", dtype=torch.int8)
            st["scale"] = torch.empty(T, device="cuda")
            st["y"] = torch.empty(T, N, device="cuda", dtype=dt)
            return st
        st["mean"] = torch.empty(T, device="cuda")
        st["rstd"] = torch.empty(T, device="cuda")
        if case["out"] == "e4m3":
            st["q"] = torch.empty(T, d, device="cuda", dtype=torch.float8_e4m3fn)
            st["scale"] = torch.empty(T, device="cuda")
        else:
            st["y"] = torch.empty_like(st["x"])
        return st
    if case["op"] == "checkpoint":
        st["x"] = (normal(case["T"], case["d"]) * loud(case["d"])).to(dt)
        return st
    M, N, K = case["M"], case["N"], case["K"]
    st["bias"] = normal(N, std=0.1)
    st["col_scale"] = normal(N, std=0.0015, mean=1.0)
    if case["op"] == "product":
        r = case["r"]
        st["x"], st["row_scale"] = _pack(normal(M, K), 0)
        st["w"], st["w_scale"] = _pack(normal(N, K, std=K ** -0.5), 0)
        st["s"] = 0.5
        st["t"] = normal(M, r, dtype=dt) if r else None
        st["b"] = normal(N, r, std=0.02, dtype=dt) if r else None
        st["residual"] = normal(M, N, dtype=dt) if case["residual"] else None
        st["y"] = torch.empty(M, N, device="cuda", dtype=dt)
        st["u"] = torch.empty(M, N, device="cuda", dtype=dt) if case["save"] else None
        return st
    x = normal(M, K, dtype=dt)
    w = normal(N, K, std=K ** -0.5, dtype=dt)
    u = torch.mm(x, w.t())
    st["dy"] = normal(M, N, dtype=dt)
    for name, v, group in (("u", u, case["u8"]), ("x", x, case["x8"] if case["dw"] else None),
                           ("w", w, (0 if case["w8"] else -1) if case["dx"] else None)):
        if group is None:
            st[name] = st[name + "_scale"] = None   # not read
        elif group < 0:
            st[name], st[name + "_scale"] = v, None
        else:
            st[name], st[name + "_scale"] = _pack(v.float(), group)
    return st


def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * 0.5 ** 0.5))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh((2 / math.pi) ** 0.5 * (z + 0.044715 * z * z * z)))
    return z


def _slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * 0.5 ** 0.5)) + z * torch.exp(-0.5 * z * z) * (2 * math.pi) ** -0.5
    if act == "gelu_tanh":
        k = (2 / math.pi) ** 0.5
        th = torch.tanh(k * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + th) + 0.5 * z * (1 - th * th) * k * (1 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


def _own(st):
    from dora_weight_norm_amd import binding as bnd

    c = st["case"]
    if c["op"] == "norm":
        if c["out"] == "e4m3":
            q, scale, h, mean, rstd = bnd.dora_layer_norm_quant(
                st["x"], st["weight"], st["norm_bias"], st["eps"], q_dtype=torch.float8_e4m3fn,
                residual=st["residual"], q=st["q"], scale=st["scale"], h=st["h"], mean=st["mean"], rstd=st["rstd"])
            return {"q": q, "scale": scale, "h": h, "mean": mean, "rstd": rstd}
        y, h, mean, rstd = bnd.dora_layer_norm(st["x"], st["weight"], st["norm_bias"], st["eps"],
                                               residual=st["residual"], y=st["y"], h=st["h"], mean=st["mean"],
                                               rstd=st["rstd"])
        return {"y": y, "h": h, "mean": mean, "rstd": rstd}
    if c["op"] == "norm_backward":
        dx, dweight, dbias = bnd.dora_layer_norm_backward(st["dy"], st["h"], st["mean"], st["rstd"], st["weight"],
                                                          dh=st["dh"], dx=st["dx"])
        return {"dx": dx, "dweight": dweight, "dbias": dbias}
    if c["op"] == "norm_product":
        q, scale, h, _, _ = bnd.dora_layer_norm_quant(
            st["x"], st["weight"], st["norm_bias"], st["eps"], q_dtype=torch.int8, residual=st["residual"],
            q=st["q"], scale=st["scale"], h=st["h"], want_stats=False)
        y, _ = bnd.dora_matmul_int8(q, st["w"], scale, st["w_scale"], col_scale=st["col_scale"], bias=st["bias"],
                                    act=c["act"], out_dtype=st["dt"], y=st["y"])
        return {"y": y, "h": h, "scale": scale}
    if c["op"] == "product":
        y, u = bnd.dora_matmul_int8(st["x"], st["w"], st["row_scale"], st["w_scale"], col_scale=st["col_scale"],
                                    t=st["t"], b=st["b"], s=st["s"], bias=st["bias"], act=c["act"],
                                    residual=st["residual"], out_dtype=st["dt"], save=c["save"], y=st["y"],
                                    u=st["u"])
        return {"y": y, "u": u} if c["save"] else {"y": y}
    if c["op"] == "checkpoint":
        q, scale = bnd.dora_quantize_rows(st["x"], group=c["group"])
        return {"x": bnd.dora_dequantize_rows(q, scale, group=c["group"], dtype=st["dt"]), "scale": scale}

    def operand(name, group):
        scale = st[name + "_scale"]
        return st[name] if scale is None else bnd.Int8Rows(st[name], scale, group)

    dx, dw, dbias, dcol, _ = bnd.dora_matmul_backward_int8(
        st["dy"], operand("u", c["u8"]), operand("x", c["x8"]), operand("w", 0), col_scale=st["col_scale"],
        bias=st["bias"], act=c["act"], need_dx=c["dx"], need_dw=c["dw"])
    return {k: v for k, v in {"dx": dx, "dw": dw, "dbias": dbias, "dcol_scale": dcol}.items() if v is not None}


def run(st):
    if own:
        return _own(st)
    c, dt = st["case"], st["dt"]
    if c["op"] in ("norm", "norm_product"):
        h = st["x"].float() + st["residual"].float()
        mean = torch.mean(h, 1)
        v = h - mean[:, None]
        rstd = 1 / torch.sqrt(torch.mean(v * v, 1) + st["eps"])
        n = v * rstd[:, None] * st["weight"] + st["norm_bias"]
        if c["op"] == "norm_product":
            q, scale = _pack(n, 0)
            u = torch.mm(q.float(), st["w"].float().t()) * scale[:, None] * st["w_scale"]
            return {"y": _act(st["col_scale"] * u + st["bias"], c["act"]).to(dt), "h": h.to(dt), "scale": scale}
        if c["out"] == "e4m3":
            q, scale = _rows_in_e4m3(n)
            return {"q": q, "scale": scale, "h": h.to(dt), "mean": mean, "rstd": rstd}
        return {"y": n.to(dt), "h": h.to(dt), "mean": mean, "rstd": rstd}
    if c["op"] == "norm_backward":
        dy, rstd = st["dy"].float(), st["rstd"][:, None]
        n = (st["h"].float() - st["mean"][:, None]) * rstd
        a = dy * st["weight"]
        dx = rstd * (a - torch.mean(a, 1, keepdim=True) - n * torch.mean(a * n, 1, keepdim=True)) + st["dh"].float()
        return {"dx": dx.to(dt), "dweight": torch.sum((dy * n).double(), 0).float(),
                "dbias": torch.sum(dy.double(), 0).float()}
    if c["op"] == "product":
        u = torch.mm(st["x"].float(), st["w"].float().t()) * st["row_scale"][:, None] * st["w_scale"]
        if st["t"] is not None:
            u = u + st["s"] * torch.mm(st["t"].float(), st["b"].float().t())
        y = _act(st["col_scale"] * u + st["bias"], c["act"])
        if st["residual"] is not None:
            y = y + st["residual"].float()
        return {"y": y.to(dt), "u": u.to(dt)} if c["save"] else {"y": y.to(dt)}
    if c["op"] == "checkpoint":
        q, scale = _pack(st["x"].float(), c["group"])
        return {"x": _unpack(q, scale, c["group"]).to(dt), "scale": scale}

    def operand(name, group):
        scale = st[name + "_scale"]
        return st[name].float() if scale is None else _unpack(st[name], scale, group)

    u = operand("u", c["u8"])
    dz = st["dy"].float() * _slope(st["col_scale"] * u + st["bias"], c["act"])
    du = st["col_scale"] * dz
    out = {"dbias": torch.sum(dz.double(), 0).float(), "dcol_scale": torch.sum((dz * u).double(), 0).float()}
    if c["dx"]:
        out["dx"] = torch.mm(du, operand("w", 0)).to(dt)
    if c["dw"]:
        out["dw"] = torch.mm(du.t(), operand("x", c["x8"])).to(dt)
    return out


def _held(rows, cols, e, group):
    """Bytes of an operand in the storage type (group < 0) or as int8 rows."""
    if group < 0:
        return rows * cols * e
    return rows * cols + 4 * rows * (-(-cols // group) if group else 1)


def work(case):
    e = {"bf16": 2, "f16": 2, "f32": 4}[case["dtype"]]
    op = case["op"]
    if op in ("norm", "norm_backward", "norm_product", "checkpoint"):
        T, d = case["T"], case["d"]
    if op == "norm":
        out = T * d + 4 * T if case["out"] == "e4m3" else T * d * e
        # x, residual, h; the output; weight, bias; mean, rstd
        return {"bytes": 3 * T * d * e + out + 8 * d + 8 * T, "flops": 8 * T * d}
    if op == "norm_backward":
        # dy, h, dh, dx; weight, dweight, dbias; mean, rstd
        return {"bytes": 4 * T * d * e + 12 * d + 8 * T, "flops": 12 * T * d}
    if op == "norm_product":
        N = case["N"]
        # x, residual, h; weight, bias; the rows and back; w and its scales; column scale and bias; y
        return {"bytes": 3 * T * d * e + 8 * d + 2 * (T * d + 4 * T) + N * d + 12 * N + T * N * e,
                "flops": 8 * T * d + 2 * T * N * d}
    if op == "checkpoint":
        # x, the packed rows and back, the restored x
        return {"bytes": 2 * T * d * e + 2 * _held(T, d, e, case["group"]), "flops": 4 * T * d}
    M, N, K = case["M"], case["N"], case["K"]
    if op == "product":
        r = case["r"]
        outs = 1 + int(case["residual"]) + int(case["save"])
        return {"bytes": (M + N) * (K + r * e) + outs * M * N * e + 12 * N + 4 * M, "flops": 2 * M * N * (K + r)}
    # dy, u; w and dx; x and dw; bias, col_scale and their gradients
    nbytes = M * N * e + _held(M, N, e, case["u8"]) + 16 * N
    flops = 0
    if case["dx"]:
        nbytes += _held(N, K, e, 0 if case["w8"] else -1) + M * K * e
        flops += 2 * M * N * K
    if case["dw"]:
        nbytes += _held(M, K, e, case["x8"]) + N * K * e
        flops += 2 * M * N * K
    return {"bytes": nbytes, "flops": flops}


def exact(case, seed):
    """The operators' definitions in 64 bits. A scale is held in 32 bits: it is rounded to them before a value is
    divided by it."""
    st = prepare(case, seed)
    f = {k: v.double() for k, v in st.items() if isinstance(v, torch.Tensor)}

    def columns(scale, d, group):   # a group's scale at each of its columns
        return scale.reshape(len(scale), -1).repeat_interleave(group or d, 1)[:, :d]

    def whole(v, top, group):       # (values as whole steps, their scale)
        scale = (top / INT8_MAX).float().double()
        return torch.round(v / columns(scale, v.shape[1], group)), scale

    def phi(z):
        return torch.special.ndtr(z)

    def squash(z):  # the tanh form of gelu is z times a logistic function of twice the inner polynomial
        return torch.sigmoid(2 * (2 / math.pi) ** 0.5 * (z + 0.044715 * z.pow(3)))

    def act(z):
        return {"none": lambda: z, "relu": lambda: z.clamp(min=0), "silu": lambda: z * torch.sigmoid(z),
                "gelu": lambda: z * phi(z), "gelu_tanh": lambda: z * squash(z)}[case["act"]]()

    if case["op"] in ("norm", "norm_product"):
        h = f["x"] + f["residual"]
        mean = h.sum(1) / case["d"]
        centred = h - mean.unsqueeze(1)
        root = (centred.pow(2).sum(1) / case["d"] + st["eps"]).sqrt()
        n = f["weight"].unsqueeze(0) * centred / root.unsqueeze(1) + f["norm_bias"].unsqueeze(0)
        top = n.abs().max(1).values
        if case["op"] == "norm_product":
            q, scale = whole(n, top, 0)
            u = (q @ f["w"].T) * scale.unsqueeze(1) * f["w_scale"].unsqueeze(0)
            return {"y": act(u * f["col_scale"] + f["bias"]), "h": h, "scale": top / INT8_MAX}
        if case["out"] != "e4m3":
            return {"y": n, "h": h, "mean": mean, "rstd": root.reciprocal()}
        # eight bits: the nearest multiple of the step 2^(e - 3), ties to the even one, e >= -6
        v = n * (E4M3_MAX / top).unsqueeze(1)
        step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
        return {"q": torch.round(v / step) * step, "scale": top / E4M3_MAX, "h": h, "mean": mean,
                "rstd": root.reciprocal()}
    if case["op"] == "norm_backward":
        n = (f["h"] - f["mean"].unsqueeze(1)) * f["rstd"].unsqueeze(1)
        a = f["dy"] * f["weight"].unsqueeze(0)
        along, level = (a * n).sum(1, keepdim=True) / case["d"], a.sum(1, keepdim=True) / case["d"]
        return {"dx": f["rstd"].unsqueeze(1) * (a - level - along * n) + f["dh"], "dweight": (f["dy"] * n).sum(0),
                "dbias": f["dy"].sum(0)}
    if case["op"] == "product":
        u = (f["x"] @ f["w"].T) * f["row_scale"].unsqueeze(1) * f["w_scale"].unsqueeze(0)
        if "t" in f:
            u = u + (st["s"] * f["t"]) @ f["b"].T
        y = act(u * f["col_scale"] + f["bias"])
        y = y + f["residual"] if "residual" in f else y
        return {"y": y, "u": u} if case["save"] else {"y": y}
    if case["op"] == "checkpoint":
        x, group = f["x"], case["group"]
        tops = [part.abs().max(1).values for part in x.split(group or case["d"], 1)]
        q, scale = whole(x, torch.stack(tops, 1), group)
        back = q * columns(scale, case["d"], group)
        return {"x": back, "scale": torch.stack(tops, 1) / INT8_MAX if group else tops[0] / INT8_MAX}

    def operand(name, group):
        scale = f.get(name + "_scale")
        return f[name] if scale is None else f[name] * columns(scale, f[name].shape[1], group)

    u = operand("u", case["u8"])
    z = u * f["col_scale"] + f["bias"]
    if case["act"] == "none":
        slope = torch.ones_like(z)
    elif case["act"] == "relu":
        slope = torch.heaviside(z, torch.zeros_like(z))
    elif case["act"] == "silu":
        slope = torch.sigmoid(z) + z * torch.sigmoid(z) * torch.sigmoid(-z)
    elif case["act"] == "gelu":
        slope = phi(z) + z * torch.exp(-z.pow(2) / 2) / math.sqrt(2 * math.pi)
    else:
        p = squash(z)
        slope = p + z * p * (1 - p) * 2 * (2 / math.pi) ** 0.5 * (1 + 3 * 0.044715 * z.pow(2))
    dz = f["dy"] * slope
    out = {"dbias": dz.sum(0), "dcol_scale": (dz * u).sum(0)}
    du = dz * f["col_scale"]
    if case["dx"]:
        out["dx"] = du @ operand("w", 0)
    if case["dw"]:
        out["dw"] = du.T @ operand("x", case["x8"])
    return out
