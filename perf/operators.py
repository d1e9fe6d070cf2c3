"""What is measured of the block around an adapted linear layer.

Two operators: the root-mean-square norm with the residual's addition (its
output in the storage type, or in 8 bits with one scale a row) and its
backward, and the matrix product with scales, a low-rank second pair, bias,
activation and residual in its epilogue, and its backward. The sizes are
those of the workloads the library is benchmarked on (8192 x 8192 at r = 384,
28672 x 8192, 4096 x 4096 at r = 64, the tiny 256 x 256), plus odd ones.

With ``own`` false, run() computes the plain form in fp32 with elementary
torch operations; with ``own`` true it calls libdora.
"""

import math

import torch

own = False

FP = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
E4M3_MAX = 448.0


def listed():
    return [
        # Decoding one sequence: the norm before a layer whose input is held in 8 bits.
        {"name": "norm one token 8 bit", "op": "norm", "dtype": "bf16", "T": 1, "d": 8192, "out": "e4m3"},
        # Prefill of 8192 tokens at the headline width, 8-bit output for the next product.
        {"name": "norm prefill 8 bit", "op": "norm", "dtype": "bf16", "T": 8192, "d": 8192, "out": "e4m3"},
        # A ragged batch at a width that no vector load divides.
        {"name": "norm ragged f16", "op": "norm", "dtype": "f16", "T": 777, "d": 3583, "out": "same"},
        # One training step's backward of the norm, 8192 tokens of a 4096-wide model.
        {"name": "norm backward", "op": "norm_backward", "dtype": "bf16", "T": 8192, "d": 4096},
        # The tiny fp32 layer (64 tokens, 256 x 256, r = 8), as tests and small experiments run it.
        {"name": "product tiny f32", "op": "product", "dtype": "f32", "M": 64, "N": 256, "K": 256, "r": 8,
         "act": "none", "residual": True, "save": False},
        # Decoding one sequence through an unmerged adapter of rank 384.
        {"name": "product one token", "op": "product", "dtype": "bf16", "M": 1, "N": 8192, "K": 8192, "r": 384,
         "act": "none", "residual": True, "save": False},
        # Decoding 16 sequences through the 8-bit MLP up projection.
        {"name": "product 16 tokens 8 bit", "op": "product", "dtype": "e4m3", "M": 16, "N": 28672, "K": 8192, "r": 0,
         "act": "silu", "residual": False, "save": False},
        # Training forward of a projection: the product is kept for the backward.
        {"name": "product training", "op": "product", "dtype": "bf16", "M": 4096, "N": 4096, "K": 4096, "r": 64,
         "act": "gelu", "residual": False, "save": True},
        # The whole adapted layer at the headline sizes: 8192 tokens, r = 384, added to the residual stream.
        {"name": "product headline", "op": "product", "dtype": "bf16", "M": 8192, "N": 8192, "K": 8192, "r": 384,
         "act": "none", "residual": True, "save": False},
        # Prefill through the 8-bit MLP up projection.
        {"name": "product prefill 8 bit", "op": "product", "dtype": "e4m3", "M": 8192, "N": 28672, "K": 8192, "r": 0,
         "act": "gelu_tanh", "residual": False, "save": False},
        # Odd sizes in fp16: no row of x or W starts on a vector boundary.
        {"name": "product ragged f16", "op": "product", "dtype": "f16", "M": 333, "N": 1001, "K": 777, "r": 24,
         "act": "relu", "residual": True, "save": False},
        # Training backward of a projection: gradients of x, W, bias and column scale.
        {"name": "product backward", "op": "product_backward", "dtype": "bf16", "M": 4096, "N": 4096, "K": 4096,
         "act": "silu"},
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
    op = rng.choice(["norm", "norm", "norm_backward", "product", "product", "product", "product_backward"])
    if op == "norm":
        return {"op": op, "dtype": rng.choice(["bf16", "bf16", "f16", "f32"]), "T": _size(rng, 1, 8192),
                "d": _size(rng, 256, 8192), "out": rng.choice(["same", "e4m3"])}
    if op == "norm_backward":
        return {"op": op, "dtype": rng.choice(["bf16", "bf16", "f16", "f32"]), "T": _size(rng, 1, 8192),
                "d": _size(rng, 256, 8192)}
    if op == "product":
        dtype = rng.choice(["bf16", "bf16", "e4m3", "e4m3", "f16", "f32"])
        top = 2048 if dtype == "f32" else 8192
        return {"op": op, "dtype": dtype, "M": _size(rng, 1, top), "N": _size(rng, 128, top),
                "K": _size(rng, 128, top), "r": 0 if dtype == "e4m3" else rng.choice([0, _size(rng, 4, 768)]),
                "act": rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]), "residual": rng.random() < 0.5,
                "save": dtype != "e4m3" and rng.random() < 0.3}
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    top = 1024 if dtype == "f32" else 8192
    return {"op": op, "dtype": dtype, "M": _size(rng, 16, top), "N": _size(rng, 128, top), "K": _size(rng, 128, top),
            "act": rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"])}


def _rows_in_8_bits(v):
    scale = v.abs().amax(1) / E4M3_MAX
    return (v / scale[:, None]).to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0, mean=0.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=gen, device="cuda") * std + mean).to(dtype)

    st = {"case": case}
    if case["op"].startswith("norm"):
        T, d, dt = case["T"], case["d"], FP[case["dtype"]]
        st["weight"] = normal(d, std=0.1, mean=1.0)
        st["eps"] = 1e-6
        # A residual stream has a few channels far larger than the rest.
        loud = torch.where(torch.rand(d, generator=gen, device="cuda") < 0.003, 20.0, 1.0)
        if case["op"] == "norm":
            st["x"] = normal(T, d, std=0.3, dtype=dt)
            st["residual"] = (normal(T, d) * loud).to(dt)
            st["h"] = torch.empty_like(st["x"])
            st["rstd"] = torch.empty(T, device="cuda")
            if case["out"] == "e4m3":
                st["q"] = torch.empty(T, d, device="cuda", dtype=torch.float8_e4m3fn)
                st["scale"] = torch.empty(T, device="cuda")
            else:
                st["y"] = torch.empty_like(st["x"])
        else:
            st["h"] = (normal(T, d) * loud).to(dt)
            st["rstd"] = (st["h"].float().square().mean(1) + st["eps"]).rsqrt()
            st["dy"] = normal(T, d, dtype=dt)
            st["dh"] = normal(T, d, dtype=dt)
            st["dx"] = torch.empty_like(st["h"])
        return st
    M, N, K = case["M"], case["N"], case["K"]
    st["bias"] = normal(N, std=0.1)
    st["col_scale"] = normal(N, std=0.0015, mean=1.0)
    if case["dtype"] == "e4m3":
        dt = torch.bfloat16
        st["x"], st["row_scale"] = _rows_in_8_bits(normal(M, K))
        st["w"], w_scale = _rows_in_8_bits(normal(N, K, std=K ** -0.5))
        st["col_scale"] = st["col_scale"] * w_scale
    else:
        dt = FP[case["dtype"]]
        st["x"] = normal(M, K, dtype=dt)
        st["w"] = normal(N, K, std=K ** -0.5, dtype=dt)
        st["row_scale"] = None
    st["dt"] = dt
    if case["op"] == "product":
        r = case["r"]
        st["s"] = 0.5
        st["t"] = normal(M, r, dtype=dt) if r else None
        st["b"] = normal(N, r, std=0.02, dtype=dt) if r else None
        st["residual"] = normal(M, N, dtype=dt) if case["residual"] else None
        st["y"] = torch.empty(M, N, device="cuda", dtype=dt)
        st["u"] = torch.empty(M, N, device="cuda", dtype=dt) if case["save"] else None
    else:
        st["u"] = torch.mm(st["x"], st["w"].t())
        st["dy"] = normal(M, N, dtype=dt)
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
            q, scale, h, rstd = bnd.dora_rms_norm_quant(st["x"], st["weight"], st["eps"], residual=st["residual"],
                                                        q=st["q"], scale=st["scale"], h=st["h"], rstd=st["rstd"])
            return {"q": q, "scale": scale, "h": h, "rstd": rstd}
        y, h, rstd = bnd.dora_rms_norm(st["x"], st["weight"], st["eps"], residual=st["residual"], y=st["y"],
                                       h=st["h"], rstd=st["rstd"])
        return {"y": y, "h": h, "rstd": rstd}
    if c["op"] == "norm_backward":
        dx, dweight = bnd.dora_rms_norm_backward(st["dy"], st["h"], st["rstd"], st["weight"], dh=st["dh"],
                                                 dx=st["dx"])
        return {"dx": dx, "dweight": dweight}
    if c["op"] == "product":
        y, u = bnd.dora_matmul(st["x"], st["w"], row_scale=st["row_scale"], col_scale=st["col_scale"], t=st["t"],
                               b=st["b"], s=st["s"], bias=st["bias"], act=c["act"], residual=st["residual"],
                               y=st["y"], u=st["u"], out_dtype=st["dt"], save=c["save"])
        return {"y": y, "u": u} if c["save"] else {"y": y}
    dx, dw, dbias, dcol, _ = bnd.dora_matmul_backward(st["dy"], st["u"], st["x"], st["w"], col_scale=st["col_scale"],
                                                      bias=st["bias"], act=c["act"])
    return {"dx": dx, "dw": dw, "dbias": dbias, "dcol_scale": dcol}


def run(st):
    if own:
        return _own(st)
    c = st["case"]
    if c["op"] == "norm":
        h = st["x"].float() + st["residual"].float()
        rstd = 1 / torch.sqrt(torch.mean(h * h, 1) + st["eps"])
        n = h * rstd[:, None] * st["weight"]
        if c["out"] == "e4m3":
            scale = n.abs().amax(1) / E4M3_MAX
            scale = torch.where(scale == 0, torch.ones_like(scale), scale)
            q = (n / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
            return {"q": q, "scale": scale, "h": h.to(st["x"].dtype), "rstd": rstd}
        return {"y": n.to(st["x"].dtype), "h": h.to(st["x"].dtype), "rstd": rstd}
    if c["op"] == "norm_backward":
        dy, rstd = st["dy"].float(), st["rstd"][:, None]
        n = st["h"].float() * rstd
        a = dy * st["weight"]
        dx = rstd * (a - n * torch.mean(a * n, 1, keepdim=True)) + st["dh"].float()
        return {"dx": dx.to(st["h"].dtype), "dweight": torch.sum((dy * n).double(), 0).float()}
    if c["op"] == "product":
        u = torch.mm(st["x"].float(), st["w"].float().t())
        if st["row_scale"] is not None:
            u = u * st["row_scale"][:, None]
        if st["t"] is not None:
            u = u + st["s"] * torch.mm(st["t"].float(), st["b"].float().t())
        y = _act(st["col_scale"] * u + st["bias"], c["act"])
        if st["residual"] is not None:
            y = y + st["residual"].float()
        return {"y": y.to(st["dt"]), "u": u.to(st["dt"])} if c["save"] else {"y": y.to(st["dt"])}
    u = st["u"].float()
    dz = st["dy"].float() * _slope(st["col_scale"] * u + st["bias"], c["act"])
    du = st["col_scale"] * dz
    return {"dx": torch.mm(du, st["w"].float()).to(st["dt"]), "dw": torch.mm(du.t(), st["x"].float()).to(st["dt"]),
            "dbias": torch.sum(dz.double(), 0).float(), "dcol_scale": torch.sum((dz * u).double(), 0).float()}


def work(case):
    e = {"bf16": 2, "f16": 2, "f32": 4, "e4m3": 1}[case["dtype"]]
    if case["op"] == "norm":
        T, d = case["T"], case["d"]
        out = T * d + 4 * T if case["out"] == "e4m3" else T * d * e
        # x, residual, h; the output; weight; rstd
        return {"bytes": 3 * T * d * e + out + 4 * d + 4 * T, "flops": 5 * T * d}
    if case["op"] == "norm_backward":
        T, d = case["T"], case["d"]
        # dy, h, dh, dx; weight, dweight; rstd
        return {"bytes": 4 * T * d * e + 8 * d + 4 * T, "flops": 10 * T * d}
    M, N, K = case["M"], case["N"], case["K"]
    o = 2 if case["dtype"] == "e4m3" else e
    if case["op"] == "product":
        r = case["r"]
        outs = 1 + int(case["residual"]) + int(case["save"])
        rows = 4 * M if case["dtype"] == "e4m3" else 0
        return {"bytes": (M + N) * (K + r) * e + outs * M * N * o + 8 * N + rows, "flops": 2 * M * N * (K + r)}
    # dy, u; x and dx; W and dw; bias, col_scale and their gradients
    return {"bytes": 2 * M * N * e + 2 * M * K * e + 2 * N * K * e + 16 * N, "flops": 4 * M * N * K}


def exact(case, seed):
    """The operators' definitions in 64 bits."""
    st = prepare(case, seed)
    f = {k: v.double() for k, v in st.items() if isinstance(v, torch.Tensor)}
    if case["op"] == "norm":
        h = f["x"] + f["residual"]
        root = (h.pow(2).sum(1) / case["d"] + st["eps"]).sqrt()
        n = f["weight"].unsqueeze(0) * h / root.unsqueeze(1)
        if case["out"] != "e4m3":
            return {"y": n, "h": h, "rstd": root.reciprocal()}
        top = n.abs().max(1).values
        # eight bits: the nearest multiple of the step 2^(e - 3), ties to the even one, e >= -6
        v = n * (E4M3_MAX / top).unsqueeze(1)
        step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
        return {"q": torch.round(v / step) * step, "scale": top / E4M3_MAX, "h": h, "rstd": root.reciprocal()}
    if case["op"] == "norm_backward":
        n = f["h"] * f["rstd"].unsqueeze(1)
        a = f["dy"] * f["weight"].unsqueeze(0)
        along = (a * n).sum(1, keepdim=True) / case["d"]
        return {"dx": f["rstd"].unsqueeze(1) * (a - along * n) + f["dh"], "dweight": (f["dy"] * n).sum(0)}

    def phi(z):
        return torch.special.ndtr(z)

    def squash(z):  # the tanh form of gelu is z times a logistic function of twice the inner polynomial
        return torch.sigmoid(2 * (2 / math.pi) ** 0.5 * (z + 0.044715 * z.pow(3)))

    if case["op"] == "product":
        u = f["x"] @ f["w"].T
        if "row_scale" in f:
            u = u * f["row_scale"].unsqueeze(1)
        if "t" in f:
            u = u + (st["s"] * f["t"]) @ f["b"].T
        z = u * f["col_scale"] + f["bias"]
        y = {"none": lambda: z, "relu": lambda: z.clamp(min=0), "silu": lambda: z * torch.sigmoid(z),
             "gelu": lambda: z * phi(z), "gelu_tanh": lambda: z * squash(z)}[case["act"]]()
        y = y + f["residual"] if "residual" in f else y
        return {"y": y, "u": u} if case["save"] else {"y": y}
    z = f["u"] * f["col_scale"] + f["bias"]
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
    du = dz * f["col_scale"]
    return {"dx": du @ f["w"], "dw": du.T @ f["x"], "dbias": dz.sum(0), "dcol_scale": (dz * f["u"]).sum(0)}
