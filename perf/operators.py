"""The measured cases of the gated feed-forward block and of the 4-bit matrix products.

Four operators, each in its plain form (elementary torch operations in 32 bits, rounded once at
the end) and as the framework's own call:

ffn_forward   out = W_down (SiLU(W_up x) * (W_gate x)); a training call also returns the
              pre-activations u = W_up x and g = W_gate x
ffn_backward  the gradients of that block for x and the three weights, from dout, x, u and g
matvec        out = W x for a few tokens, W held as 4-bit codes with a scale (and possibly a zero
              point) per group of consecutive columns: w = scale * (code - zero)
experts       the routed experts of the layer for a few tokens, every expert's three matrices in
              4 bits: out_t = sum_j w_tj W_down^e SwiGLU(W_up^e x_t, W_gate^e x_t), e = ids[t, j]
"""
import math

import torch

own = False

# sizes of the repository's configurations: hidden 2048 / inter 512 (the decode layer, 256
# experts, top-8), 2048 / 2048 (64 experts, top-2), 4096 / 1536 (16384 tokens), 7168 / 2048
# (4096 tokens, shared expert)


def listed():
    return [
        # one token through the dense block of a small layer: latency is all there is
        {"name": "ffn fwd 1 token 2048x512", "op": "ffn_forward", "T": 1, "H": 2048, "D": 512, "train": False},
        # a decode batch through the largest layer's shared expert: every weight read once
        {"name": "ffn fwd 16 tokens 7168x2048", "op": "ffn_forward", "T": 16, "H": 7168, "D": 2048, "train": False},
        # a ragged prefill chunk: too few rows to fill the GPU with large tiles
        {"name": "ffn fwd 333 tokens 2048x2048", "op": "ffn_forward", "T": 333, "H": 2048, "D": 2048, "train": False},
        # a training batch through the largest layer's shared expert, keeping u and g
        {"name": "ffn train 4096 tokens 7168x2048", "op": "ffn_forward", "T": 4096, "H": 7168, "D": 2048, "train": True},
        # a short, odd micro-batch's gradients
        {"name": "ffn bwd 515 tokens 2048x512", "op": "ffn_backward", "T": 515, "H": 2048, "D": 512},
        # the gradients of that training batch
        {"name": "ffn bwd 4096 tokens 7168x2048", "op": "ffn_backward", "T": 4096, "H": 7168, "D": 2048},
        # the longest batch of the configurations
        {"name": "ffn bwd 16384 tokens 4096x1536", "op": "ffn_backward", "T": 16384, "H": 4096, "D": 1536},
        # one token times one projection, 4 bits symmetric
        {"name": "matvec 1 token 2048x7168 g128", "op": "matvec", "T": 1, "R": 2048, "K": 7168, "group": 128, "zeros": False, "out": "float32"},
        # five tokens (a speculative step), an odd number of rows, a ragged last group, zero points
        {"name": "matvec 5 tokens 8193x2056 g64", "op": "matvec", "T": 5, "R": 8193, "K": 2056, "group": 64, "zeros": True, "out": "bfloat16"},
        # one token through the decode layer's experts
        {"name": "experts 1 token 2048x512 e256", "op": "experts", "T": 1, "H": 2048, "D": 512, "E": 256, "k": 8, "group": 128, "zeros": False},
        # the decode batch, finer groups with zero points
        {"name": "experts 16 tokens 2048x512 e256", "op": "experts", "T": 16, "H": 2048, "D": 512, "E": 256, "k": 8, "group": 32, "zeros": True},
        # a decode batch over one GPU's share of the largest layer's experts
        {"name": "experts 8 tokens 7168x2048 e64", "op": "experts", "T": 8, "H": 7168, "D": 2048, "E": 64, "k": 8, "group": 128, "zeros": False},
    ]


def _log(rng, lo, hi, step=1):
    return max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi))) // step * step))


def draw(rng):
    op = rng.choice(["ffn_forward", "ffn_backward", "matvec", "experts"])
    if op in ("ffn_forward", "ffn_backward"):
        H, D = _log(rng, 128, 7168, 8), _log(rng, 64, 4096, 8)
        most = {"ffn_forward": 4096 * 7168 * 2048, "ffn_backward": 16384 * 4096 * 1536}[op]
        T = _log(rng, 1, min(16384, max(2, most // (H * D))))
        c = {"op": op, "T": T, "H": H, "D": D}
        if op == "ffn_forward":
            c["train"] = rng.random() < 0.5
        return c
    if op == "matvec":
        return {"op": op, "T": _log(rng, 1, 16), "R": _log(rng, 33, 16384), "K": _log(rng, 128, 7168, 8),
                "group": rng.choice([32, 64, 128]), "zeros": rng.random() < 0.5, "out": rng.choice(["float32", "bfloat16"])}
    E = _log(rng, 4, 128)
    k = rng.randint(1, min(8, E))
    return {"op": op, "T": _log(rng, 1, max(2, min(16, 64 // k))), "H": _log(rng, 256, 4096, 16), "D": _log(rng, 128, 2048, 16), "E": E, "k": k,
            "group": rng.choice([32, 64, 128]), "zeros": rng.random() < 0.5}


def _normal(shape, sigma, gen, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=gen, device="cuda") * sigma).to(dtype)


def _codes(rows, cols, group, zeros, gen):
    """A quantised matrix as a checkpoint holds it: two codes a byte (the even column in the low
    half), and per row and group a bf16 scale and, where asked, a zero point (else 8)."""
    # codes that crowd around the middle, as those of normal weights do
    b = torch.randint(0, 256, (rows, cols), generator=gen, device="cuda", dtype=torch.uint8)
    b = ((b & 15) + (b >> 4)) >> 1
    q = b[:, 0::2] | (b[:, 1::2] << 4)
    g = (cols + group - 1) // group
    s = torch.rand((rows, g), generator=gen, device="cuda") * 0.5 + 0.75
    s = (s * (0.3 / math.sqrt(cols))).to(torch.bfloat16)
    z = torch.randint(6, 10, (rows, g), generator=gen, device="cuda", dtype=torch.uint8) if zeros else None
    return {"q": q, "s": s, "z": z}


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    c, s = case, {"case": case}
    if c["op"] in ("ffn_forward", "ffn_backward"):
        T, H, D = c["T"], c["H"], c["D"]
        s["x"] = _normal((T, H), 1.0, gen)
        s["w"] = {"Ws_up": _normal((D, H), 0.9 / math.sqrt(H), gen), "Ws_gate": _normal((D, H), 0.9 / math.sqrt(H), gen),
                  "Ws_down": _normal((H, D), 0.9 / math.sqrt(D), gen)}
        if c["op"] == "ffn_backward":  # u and g as the forward of the training step left them
            s["dout"] = _normal((T, H), 1.0, gen)
            s["u"] = (s["x"].float() @ s["w"]["Ws_up"].float().t()).to(torch.bfloat16)
            s["g"] = (s["x"].float() @ s["w"]["Ws_gate"].float().t()).to(torch.bfloat16)
        if own:
            from mixture_experts_layer_block_b200.native import MoELayer
            s["layer"] = MoELayer(hidden=H, inter=D, num_experts=1, top_k=1, block_m=16, max_tokens=1)
        return s
    if c["op"] == "matvec":
        s["x"] = _normal((c["T"], c["K"]), 1.0, gen)
        s["w"] = _codes(c["R"], c["K"], c["group"], c["zeros"], gen)
        if own:
            from mixture_experts_layer_block_b200.native import MoELayer
            s["layer"] = MoELayer(hidden=c["K"], inter=8, num_experts=1, top_k=1, block_m=16, max_tokens=1)
            s["packed"] = s["layer"].pack_int4(s["w"]["q"], s["w"]["s"], s["w"]["z"], c["group"])
        return s
    T, H, D, E, k = c["T"], c["H"], c["D"], c["E"], c["k"]
    s["x"] = _normal((T, H), 1.0, gen)
    s["w"] = {"W_up": _codes(E * D, H, c["group"], c["zeros"], gen), "W_gate": _codes(E * D, H, c["group"], c["zeros"], gen),
              "W_down": _codes(E * H, D, c["group"], c["zeros"], gen)}
    # a softmax over the k experts that a router with unequal favourites picks
    logits = torch.randn((T, E), generator=gen, device="cuda") + torch.randn((1, E), generator=gen, device="cuda")
    top = torch.topk(logits, k, dim=1)
    s["ids"], s["p"] = top.indices.to(torch.int32), torch.softmax(top.values, dim=1)
    if own:
        from mixture_experts_layer_block_b200.native import MoELayer
        s["layer"] = MoELayer(hidden=H, inter=D, num_experts=E, top_k=k, block_m=16, max_tokens=16)
        s["packed"] = {n: s["layer"].pack_int4(w["q"], w["s"], w["z"], c["group"]) for n, w in s["w"].items()}
    return s


def _own(s):
    c, layer, x = s["case"], s["layer"], s["x"]
    if c["op"] == "ffn_forward":
        out = torch.empty_like(x)
        if not c["train"]:
            return {"out": layer.ffn_forward(x, s["w"], out)}
        u = torch.empty((c["T"], c["D"]), dtype=torch.bfloat16, device="cuda")
        g = torch.empty_like(u)
        layer.ffn_forward(x, s["w"], out, u=u, g=g)
        return {"out": out, "u": u, "g": g}
    if c["op"] == "ffn_backward":
        grads = {"x": torch.empty_like(x), **{n: torch.empty_like(w) for n, w in s["w"].items()}}
        layer.ffn_backward(s["dout"], x, s["u"], s["g"], s["w"], grads)
        return grads
    if c["op"] == "matvec":
        out = torch.empty((c["T"], c["R"]), dtype=getattr(torch, c["out"]), device="cuda")
        return {"out": layer.matvec_int4(x, s["packed"], out)}
    return {"out": layer.experts_int4(x, s["ids"], s["p"], s["packed"], torch.empty_like(x))}


def _matrix(q, s, z, group):
    """The fp32 values of packed codes [..., rows, cols / 2] with scales [..., rows, groups]."""
    code = torch.stack((q & 15, q >> 4), dim=-1).flatten(-2).float()
    at = torch.arange(code.shape[-1], device=code.device) // group
    return (code - (8.0 if z is None else z.float()[..., at])) * s.float()[..., at]


def run(s):
    if own:
        return _own(s)
    c, x, w = s["case"], s["x"].float(), s["w"]
    if c["op"] == "ffn_forward":
        u, g = x @ w["Ws_up"].float().t(), x @ w["Ws_gate"].float().t()
        out = ((u / (1 + torch.exp(-u))) * g) @ w["Ws_down"].float().t()
        if not c["train"]:
            return {"out": out.to(torch.bfloat16)}
        return {"out": out.to(torch.bfloat16), "u": u.to(torch.bfloat16), "g": g.to(torch.bfloat16)}
    if c["op"] == "ffn_backward":
        u, g, dout = s["u"].float(), s["g"].float(), s["dout"].float()
        sig = 1 / (1 + torch.exp(-u))
        dh = dout @ w["Ws_down"].float()
        du, dg = dh * g * (sig * (1 + u * (1 - sig))), dh * (u * sig)
        grads = {"x": du @ w["Ws_up"].float() + dg @ w["Ws_gate"].float(), "Ws_up": du.t() @ x, "Ws_gate": dg.t() @ x,
                 "Ws_down": dout.t() @ (u * sig * g)}
        return {n: v.to(torch.bfloat16) for n, v in grads.items()}
    if c["op"] == "matvec":
        return {"out": (x @ _matrix(w["q"], w["s"], w["z"], c["group"]).t()).to(getattr(torch, c["out"]))}
    T, H, D, E, k = c["T"], c["H"], c["D"], c["E"], c["k"]
    ids = s["ids"].long().flatten()

    def picked(m, rows, cols):  # [T*k, rows, cols]: the matrices of the chosen experts
        z = m["z"]
        return _matrix(m["q"].view(E, rows, cols // 2)[ids], m["s"].view(E, rows, -1)[ids],
                       None if z is None else z.view(E, rows, -1)[ids], c["group"])

    xs = x.repeat_interleave(k, dim=0).unsqueeze(2)
    u = torch.bmm(picked(w["W_up"], D, H), xs)
    g = torch.bmm(picked(w["W_gate"], D, H), xs)
    y = torch.bmm(picked(w["W_down"], H, D), (u / (1 + torch.exp(-u))) * g).view(T, k, H)
    return {"out": (y * s["p"].unsqueeze(2)).sum(dim=1).to(torch.bfloat16)}


def work(case):
    c = case
    if c["op"] in ("ffn_forward", "ffn_backward"):
        T, H, D = c["T"], c["H"], c["D"]
        if c["op"] == "ffn_forward":
            return {"bytes": 2 * (2 * T * H + 3 * H * D + (2 * T * D if c["train"] else 0)), "flops": 6 * T * H * D}
        return {"bytes": 2 * (3 * T * H + 2 * T * D + 6 * H * D), "flops": 12 * T * H * D}

    def held(rows, cols):  # codes, scales and zero points
        return rows * cols / 2 + rows * -(-cols // c["group"]) * (3 if c["zeros"] else 2)

    if c["op"] == "matvec":
        return {"bytes": held(c["R"], c["K"]) + 2 * c["T"] * c["K"] + c["T"] * c["R"] * (4 if c["out"] == "float32" else 2),
                "flops": 2 * c["T"] * c["R"] * c["K"]}
    T, H, D, E, k = c["T"], c["H"], c["D"], c["E"], c["k"]
    # about how many experts the tokens reach: the mean over a few draws of prepare's router
    gen, hit = torch.Generator().manual_seed(0), 0.0
    for _ in range(8):
        logits = torch.randn((T, E), generator=gen) + torch.randn((1, E), generator=gen)
        hit += torch.topk(logits, k, dim=1).indices.unique().numel() / 8
    return {"bytes": hit * (2 * held(D, H) + held(H, D)) + 4 * T * H + 8 * T * k, "flops": 6 * T * k * H * D}


def exact(case, seed):
    """The same outputs by the operators' definitions in 64 bits, one expert (or row block) at a time."""
    c, s = case, prepare(case, seed)
    x = s["x"].double()

    def block(u, g):
        return u * torch.sigmoid(u) * g

    if c["op"] == "ffn_forward":
        up, gate, down = (s["w"][n].double() for n in ("Ws_up", "Ws_gate", "Ws_down"))
        u, g = torch.einsum("th,dh->td", x, up), torch.einsum("th,dh->td", x, gate)
        out = torch.einsum("td,hd->th", block(u, g), down)
        return {"out": out, "u": u, "g": g} if c["train"] else {"out": out}
    if c["op"] == "ffn_backward":
        up, gate, down = (s["w"][n].double() for n in ("Ws_up", "Ws_gate", "Ws_down"))
        u, g, dout = s["u"].double(), s["g"].double(), s["dout"].double()
        u.requires_grad_(True)
        g.requires_grad_(True)
        h = block(u, g)
        du, dg = torch.autograd.grad(h, (u, g), torch.einsum("th,hd->td", dout, down))
        return {"x": torch.einsum("td,dh->th", du, up) + torch.einsum("td,dh->th", dg, gate), "Ws_up": torch.einsum("td,th->dh", du, x),
                "Ws_gate": torch.einsum("td,th->dh", dg, x), "Ws_down": torch.einsum("th,td->hd", dout, h.detach())}

    def values(m, r0, r1):
        """Rows r0..r1 of a quantised matrix in fp64."""
        q = m["q"][r0:r1]
        v = torch.empty((r1 - r0, 2 * q.shape[1]), dtype=torch.float64, device=q.device)
        v[:, 0::2], v[:, 1::2] = (q % 16).double(), (q // 16).double()
        for i in range(m["s"].shape[1]):
            part = v[:, i * c["group"]:(i + 1) * c["group"]]
            part -= 8 if m["z"] is None else m["z"][r0:r1, i:i + 1].double()
            part *= m["s"][r0:r1, i:i + 1].double()
        return v

    if c["op"] == "matvec":
        return {"out": x @ values(s["w"], 0, c["R"]).t()}
    out = torch.zeros((c["T"], c["H"]), dtype=torch.float64, device=x.device)
    ids = s["ids"].tolist()
    for e in sorted({e for row in ids for e in row}):
        up, gate = (values(s["w"][n], e * c["D"], (e + 1) * c["D"]) for n in ("W_up", "W_gate"))
        down = values(s["w"]["W_down"], e * c["H"], (e + 1) * c["H"])
        for t, row in enumerate(ids):
            for j, got in enumerate(row):
                if got == e:
                    out[t] += s["p"][t, j].double() * (down @ block(up @ x[t], gate @ x[t]))
    return {"out": out}
