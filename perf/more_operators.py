"""Cases of the operators between the embedding lookup and the gradient buffers,
each in a plain form (elementary torch operations) and as calls of libzq:

ce_loss      softmax cross entropy of the vocabulary projection, per token
ce_grad      its gradient: of the hidden states and of the projection
swiglu       silu(gate) * up with both inputs kept as int8 blocks, then the
             gradients from the kept blocks (one training step of the layer)
swiglu_grad  the gradients alone, with the product recomputed for the layer
             that follows
linear_grad  a linear layer's weight gradient from its input kept as int8
             blocks: written, or added (fp32)

A projection is bf16 / fp16 rows or qwZ int8 codes; a value that is held in
int8 and enters a matrix product is the code times its block's scale rounded
to the product's 16-bit type, as zq_dequant_int8 gives it.

Sizes are those of the repository's models (vocabularies 32000 and 50257;
widths 768, 2048, 4096; FFN 5632 and 11008) or generic.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
BYTES = {"fp32": 4, "bf16": 2, "fp16": 2}


def listed():
    return [
        # Scoring one token with the 7.5B model's head, as in decoding: latency and one read of the head.
        {"name": "ce_loss_1_token_bf16", "op": "ce_loss", "type": "bf16", "tokens": 1, "dim": 4096, "rows": 32000,
         "block": 0, "long": True, "pad": 0, "scale": 1.0},
        # A short evaluation batch on the 124M model's tied table: an odd vocabulary, ragged tokens, padding.
        {"name": "ce_loss_333_fp16", "op": "ce_loss", "type": "fp16", "tokens": 333, "dim": 768, "rows": 50257,
         "block": 0, "long": False, "pad": 10, "scale": 1.0},
        # The 7.5B model's micro-batch straight from what the qwZ all-gather delivered (int8, block 2048): the largest.
        {"name": "ce_loss_16384_int8_bf16", "op": "ce_loss", "type": "bf16", "tokens": 16384, "dim": 4096,
         "rows": 32000, "block": 2048, "long": True, "pad": 0, "scale": 1.0},
        # Few tokens, an odd width, a small vocabulary.
        {"name": "ce_grad_65_odd_fp16", "op": "ce_grad", "type": "fp16", "tokens": 65, "dim": 513, "rows": 1000,
         "block": 0, "long": False, "pad": 10, "scale": 0.5},
        # The ~0.85B model's micro-batch of 8 x 1024 tokens.
        {"name": "ce_grad_8192_bf16", "op": "ce_grad", "type": "bf16", "tokens": 8192, "dim": 2048, "rows": 32000,
         "block": 0, "long": True, "pad": 10, "scale": 1.0},
        # The 7.5B model's micro-batch, the head in int8: the largest.
        {"name": "ce_grad_16384_int8_bf16", "op": "ce_grad", "type": "bf16", "tokens": 16384, "dim": 4096,
         "rows": 32000, "block": 2048, "long": True, "pad": 0, "scale": 1.0},
        # One token through the ~0.85B model's FFN width: launches and latency.
        {"name": "swiglu_1_token_fp16", "op": "swiglu", "type": "fp16", "n": 5632, "block": 128},
        # The ~0.85B model's micro-batch, less one token.
        {"name": "swiglu_8191_bf16", "op": "swiglu", "type": "bf16", "n": 8191 * 5632, "block": 128},
        # The 7.5B model's backward pass: the largest.
        {"name": "swiglu_grad_16384_bf16", "op": "swiglu_grad", "type": "bf16", "n": 16384 * 11008, "block": 256},
        # Ragged sizes on every side.
        {"name": "linear_grad_odd_fp16", "op": "linear_grad", "type": "fp16", "grad": "fp16", "mode": "write",
         "tokens": 1001, "in": 515, "out": 321, "block": 64},
        # The ~0.85B model's attention output projection: a long sum over a small gradient.
        {"name": "linear_grad_8192_bf16", "op": "linear_grad", "type": "bf16", "grad": "bf16", "mode": "write",
         "tokens": 8192, "in": 2048, "out": 2048, "block": 128},
        # The 7.5B model's down projection, later micro-batches: adds into the fp32 gradient. The largest.
        {"name": "linear_grad_16384_fp32", "op": "linear_grad", "type": "bf16", "grad": "fp32", "mode": "add",
         "tokens": 16384, "in": 11008, "out": 4096, "block": 256},
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["ce_loss", "ce_loss", "ce_grad", "ce_grad", "swiglu", "swiglu_grad", "linear_grad", "linear_grad"])
    half = rng.choice(["bf16", "bf16", "fp16"])
    if op in ("swiglu", "swiglu_grad"):
        return {"op": op, "type": rng.choice([half, "fp32"]), "n": spread(1000, 1 << 26), "block": 1 << rng.randrange(5, 13)}
    if op == "linear_grad":
        c = {"op": op, "type": half, "grad": rng.choice([half, "fp32"]), "tokens": spread(16, 16384),
             "in": spread(64, 11008), "out": spread(64, 11008), "block": 1 << rng.randrange(5, 13)}
        while c["in"] * c["out"] > 11008 * 4096:
            c["in"] = max(64, c["in"] // 2)
        c["mode"] = rng.choice(["write", "add"]) if c["grad"] == "fp32" else "write"
        if rng.random() < 0.5:  # widths as models have them
            c["in"], c["out"] = -(-c["in"] // 64) * 64, -(-c["out"] // 64) * 64
        return c
    c = {"op": op, "type": half, "tokens": spread(1 if op == "ce_loss" else 32, 16384), "dim": spread(64, 4096),
         "rows": spread(100, 50257), "block": rng.choice([0, 1 << rng.randrange(5, 13)]), "long": rng.random() < 0.5,
         "pad": rng.choice([0, 10, 50]), "scale": rng.choice([1.0, 0.5])}
    if rng.random() < 0.5:
        c["dim"] = -(-c["dim"] // 64) * 64
    while c["tokens"] * c["dim"] * c["rows"] > 16384 * 4096 * 32000:
        c["tokens"] //= 2
    return c


def quantize(x, block):
    """Symmetric int8 blocks of the flat tensor: codes (whole numbers in
    float32, padded to whole blocks) and the blocks' scales."""
    flat = x.reshape(-1).float()
    v = torch.nn.functional.pad(flat, (0, -flat.numel() % block)).view(-1, block)
    s = v.abs().amax(1, keepdim=True) / 127
    k = torch.where(s > 0, torch.round(v / s).clamp(-127, 127), 0.0)
    return k, s


def values(codes, scales, block):
    """The float32 values that flat codes stand for."""
    k = torch.nn.functional.pad(codes.reshape(-1).float(), (0, -codes.numel() % block)).view(-1, block)
    return (k * scales[:, None]).view(-1)[:codes.numel()].view(codes.shape)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s, t = dict(case), TYPES[case["type"]]

    def normal(*shape, std=1.0, like=t):
        return torch.randn(*shape, generator=gen, device="cuda").mul_(std).to(like)

    def kept(*shape, block):
        """An activation as a forward pass kept it: int8 codes and scales."""
        k, scales = quantize(normal(*shape, like=torch.float32), block)
        return k.view(-1)[:math.prod(shape)].to(torch.int8).view(*shape), scales.view(-1)

    if case["op"] in ("swiglu", "swiglu_grad"):
        n, b = case["n"], case["block"]
        blocks = -(-n // b)
        s["dh"] = normal(n, std=1e-2)
        s["h"], s["dgate"], s["dup"] = (torch.empty(n, device="cuda", dtype=t) for _ in range(3))
        if case["op"] == "swiglu":
            s["gate"], s["up"] = normal(n, std=1.5), normal(n)
            s["gate_codes"], s["up_codes"] = (torch.empty(n, device="cuda", dtype=torch.int8) for _ in range(2))
            s["gate_scales"], s["up_scales"] = (torch.empty(blocks, device="cuda") for _ in range(2))
        else:
            s["gate_codes"], s["gate_scales"] = kept(n, block=b)
            s["up_codes"], s["up_scales"] = kept(n, block=b)
        return s
    if case["op"] == "linear_grad":
        n, i, o = case["tokens"], case["in"], case["out"]
        s["dy"] = normal(n, o, std=1e-2)
        s["codes"], s["scales"] = kept(n, i, block=case["block"])
        s["grad_out"] = normal(o, i, std=1e-1, like=TYPES[case["grad"]])
        if own:  # the workspace that a training program keeps beside its buffers
            from weight_communication_zero_amd import zq
            s["workspace"] = torch.empty(zq.linear_grad_workspace(n, o, i), device="cuda", dtype=torch.uint8)
        return s
    n, d, rows = case["tokens"], case["dim"], case["rows"]
    w = torch.randn(rows, d, generator=gen, device="cuda").mul_(0.02)
    ids = torch.randint(0, rows, (n,), generator=gen, device="cuda")
    # Hidden states of unit variance that lean to the token that follows, from not at all to nearly sure.
    lean = torch.rand(n, 1, generator=gen, device="cuda").mul_(14 / case["scale"])
    x = torch.randn(n, d, generator=gen, device="cuda")
    s["x"] = x.add_(w[ids] * (lean / w[ids].square().sum(1, keepdim=True))).to(t)
    left_out = torch.rand(n, generator=gen, device="cuda") * 100 < case["pad"]
    if n > 1 or case["pad"] < 50:
        left_out[0] = False
    ids = torch.where(left_out, -1, ids)
    s["ids"] = ids if case["long"] else ids.int()
    if case["block"]:
        k, scales = quantize(w, case["block"])
        s["codes"], s["scales"] = k.view(-1)[:rows * d].to(torch.int8).view(rows, d), scales.view(-1)
        del k
    else:
        s["w"] = w.to(t)
    del w
    if case["op"] == "ce_loss":
        s["loss"], s["lse"] = (torch.empty(n, device="cuda") for _ in range(2))
    else:
        # The mean over the batch with weights of the tokens; fp16 training scales its loss.
        s["dloss"] = torch.rand(n, generator=gen, device="cuda").add_(0.5).mul_((8192 if t == torch.float16 else 1) / n)
        there = ids >= 0
        z = torch.empty(n, device="cuda")
        wt = weight(s).float().t()
        for i in range(0, n, 4096):
            z[i:i + 4096] = torch.logsumexp((s["x"][i:i + 4096].float() @ wt) * case["scale"], 1)
        s["lse"] = torch.where(there, z, 0.0)
        s["dx"] = torch.empty(n, d, device="cuda", dtype=t)
        s["dw"] = torch.empty(rows, d, device="cuda", dtype=t)
    if own:
        from weight_communication_zero_amd import zq
        size = zq.ce_loss_workspace if case["op"] == "ce_loss" else zq.ce_grad_workspace
        s["workspace"] = torch.empty(size(n, rows, d), device="cuda", dtype=torch.uint8)
    return s


def weight(s):
    """The projection in the hidden states' type."""
    return values(s["codes"], s["scales"], s["block"]).to(s["x"].dtype) if s["block"] else s["w"]


def run(s):
    if own:
        return run_own(s)
    op = s["op"]
    if op in ("swiglu", "swiglu_grad"):
        out, t = {}, s["dh"].dtype
        if op == "swiglu":
            g, u = s["gate"].float(), s["up"].float()
            out["h"] = (g / (1 + torch.exp(-g)) * u).to(t)
            kept = [quantize(x, s["block"]) for x in (g, u)]
            g, u = ((k * c).view(-1)[:s["n"]] for k, c in kept)
        else:
            g, u = (values(s[x + "_codes"], s[x + "_scales"], s["block"]) for x in ("gate", "up"))
        sig, dh = 1 / (1 + torch.exp(-g)), s["dh"].float()
        silu = g * sig
        if op == "swiglu_grad":
            out["h"] = (silu * u).to(t)
        out["dgate"] = (dh * u * (sig + silu * (1 - sig))).to(t)
        out["dup"] = (dh * silu).to(t)
        return out
    if op == "linear_grad":
        x = values(s["codes"], s["scales"], s["block"]).to(s["dy"].dtype).float()
        d = s["dy"].float().t() @ x
        if s["mode"] == "add":
            s["grad_out"].add_(d)
        else:
            s["grad_out"].copy_(d)
        return {"grad": s["grad_out"]}
    x, w, ids = s["x"].float(), weight(s).float(), s["ids"].long()
    there = (ids >= 0) & (ids < s["rows"])
    at = torch.where(there, ids, 0)
    z = (x @ w.t()) * s["scale"]
    if op == "ce_loss":
        top = z.amax(1, keepdim=True)
        lse = (z - top).exp().sum(1).log() + top[:, 0]
        return {"loss": torch.where(there, lse - z.gather(1, at[:, None])[:, 0], 0.0), "lse": torch.where(there, lse, 0.0)}
    g = (z - s["lse"][:, None]).exp()
    g.scatter_add_(1, at[:, None], torch.full_like(z[:, :1], -1.0))
    g = torch.where(there[:, None], g * (s["dloss"] * s["scale"])[:, None], 0.0)
    return {"dx": (g @ w).to(s["dx"].dtype), "dw": (g.t() @ x).to(s["dw"].dtype)}


def run_own(s):
    from weight_communication_zero_amd import zq
    op = s["op"]
    if op in ("swiglu", "swiglu_grad"):
        kept = (s["gate_codes"], s["gate_scales"], s["up_codes"], s["up_scales"])
        if op == "swiglu":
            zq.zq_swiglu_int8(s["gate"], s["up"], s["block"], s["h"], *kept)
            zq.zq_swiglu_grad_int8(*kept, s["block"], s["dh"], s["dgate"], s["dup"])
        else:
            zq.zq_swiglu_grad_int8(*kept, s["block"], s["dh"], s["dgate"], s["dup"], h=s["h"])
        return {"h": s["h"], "dgate": s["dgate"], "dup": s["dup"]}
    if op == "linear_grad":
        zq.zq_linear_grad_int8(s["dy"], s["codes"], s["scales"], s["block"], s["grad_out"],
                               zq.ZQ_GRAD_ADD if s["mode"] == "add" else zq.ZQ_GRAD_WRITE, s["workspace"])
        return {"grad": s["grad_out"]}
    if op == "ce_loss":
        if s["block"]:
            zq.zq_ce_loss_int8(s["x"], s["codes"], s["scales"], s["block"], s["ids"], s["scale"], s["loss"], s["lse"],
                               s["workspace"])
        else:
            zq.zq_ce_loss(s["x"], s["w"], s["ids"], s["scale"], s["loss"], s["lse"], s["workspace"])
        return {"loss": s["loss"], "lse": s["lse"]}
    if s["block"]:
        zq.zq_ce_grad_int8(s["x"], s["codes"], s["scales"], s["block"], s["ids"], s["scale"], s["lse"], s["dloss"],
                           s["dx"], s["dw"], zq.ZQ_GRAD_WRITE, s["workspace"])
    else:
        zq.zq_ce_grad(s["x"], s["w"], s["ids"], s["scale"], s["lse"], s["dloss"], s["dx"], s["dw"], zq.ZQ_GRAD_WRITE,
                      s["workspace"])
    return {"dx": s["dx"], "dw": s["dw"]}


def work(case):
    op = case["op"]
    e = BYTES[case["type"]]
    if op in ("swiglu", "swiglu_grad"):
        n, q = case["n"], 2 * (1 + 4 / case["block"])
        if op == "swiglu":  # gate, up -> h, codes; codes, dh -> dgate, dup
            return {"bytes": n * (3 * e + q + q + 3 * e), "flops": 30 * n}
        return {"bytes": n * (q + 4 * e), "flops": 15 * n}
    if op == "linear_grad":
        n, i, o = case["tokens"], case["in"], case["out"]
        g = BYTES[case["grad"]] * (2 if case["mode"] == "add" else 1)
        return {"bytes": n * o * e + n * i * (1 + 4 / case["block"]) + o * i * g, "flops": 2 * n * i * o}
    n, d, rows = case["tokens"], case["dim"], case["rows"]
    valid = n * (1 - case["pad"] / 100)
    w = rows * d * (1 + 4 / case["block"] if case["block"] else e)
    ids = n * (8 if case["long"] else 4)
    if op == "ce_loss":
        return {"bytes": valid * d * e + w + ids + 8 * n, "flops": 2 * valid * d * rows}
    return {"bytes": valid * d * e + w + ids + 8 * n + n * d * e + rows * d * e, "flops": 6 * valid * d * rows}


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op in ("swiglu", "swiglu_grad"):
        b, n = case["block"], case["n"]
        step = (1 << 24) // b * b
        out = {k: torch.empty(n, device="cuda", dtype=torch.float64) for k in ("h", "dgate", "dup")}
        for i in range(0, n, step):
            j = min(n, i + step)
            if op == "swiglu":
                g, u = s["gate"][i:j].double(), s["up"][i:j].double()
                out["h"][i:j] = g * torch.special.expit(g) * u
                g, u = exact_kept(g, b), exact_kept(u, b)
            else:
                at = torch.arange(i, j, device="cuda") // b
                g, u = (s[x + "_codes"][i:j].double() * s[x + "_scales"].double()[at] for x in ("gate", "up"))
                out["h"][i:j] = g * torch.special.expit(g) * u
            sg, dh = torch.special.expit(g), s["dh"][i:j].double()
            out["dup"][i:j] = dh * g * sg
            out["dgate"][i:j] = dh * u * sg * (1 + g * torch.special.expit(-g))
        return out
    if op == "linear_grad":
        total = s["grad_out"].double() if case["mode"] == "add" else torch.zeros_like(s["grad_out"], dtype=torch.float64)
        for i in range(0, case["tokens"], 4096):
            at = torch.arange(i * case["in"], min(i + 4096, case["tokens"]) * case["in"], device="cuda") // case["block"]
            x = s["codes"][i:i + 4096].reshape(-1).double() * s["scales"].double()[at]
            x = x.float().to(s["dy"].dtype).double().view(-1, case["in"])
            total.addmm_(s["dy"][i:i + 4096].double().t().contiguous(), x)
        return {"grad": total}
    n, rows, dim = case["tokens"], case["rows"], case["dim"]
    if case["block"]:
        at = torch.arange(rows * dim, device="cuda") // case["block"]
        w = (s["codes"].reshape(-1).double() * s["scales"].double()[at]).float().to(s["x"].dtype).double().view(rows, dim)
        del at
    else:
        w = s["w"].double()
    ids = s["ids"].cpu().long().numpy()
    there = np.nonzero((ids >= 0) & (ids < rows))[0]
    wt = w.t().contiguous()
    if op == "ce_loss":
        loss, lse = (torch.zeros(n, device="cuda", dtype=torch.float64) for _ in range(2))
    else:
        dx, dw = torch.zeros(n, dim, device="cuda", dtype=torch.float64), torch.zeros_like(w)
    for i in range(0, len(there), 2048):
        t = torch.from_numpy(there[i:i + 2048]).cuda()
        y = torch.from_numpy(ids[there[i:i + 2048]]).cuda()
        x = s["x"][t].double()
        z = (x @ wt) * case["scale"]
        if op == "ce_loss":
            lse[t] = torch.logsumexp(z, 1)
            loss[t] = lse[t] - z[torch.arange(len(t), device="cuda"), y]
            continue
        p = torch.exp(z - s["lse"][t].double()[:, None])
        p[torch.arange(len(t), device="cuda"), y] -= 1
        p *= (s["dloss"][t].double() * case["scale"])[:, None]
        dx[t] = p @ w
        dw += p.t().contiguous() @ x
    return {"loss": loss, "lse": lse} if op == "ce_loss" else {"dx": dx, "dw": dw}


def exact_kept(x, block):
    """The values that int8 blocks hold of x: scales and quotients are rounded
    to 32 bits, by the format's definition, before the codes."""
    n = x.numel()
    v = torch.zeros(-(-n // block) * block, device="cuda", dtype=torch.float64)
    v[:n] = x
    v = v.view(-1, block)
    s = (v.abs().amax(1) / 127).float().double()[:, None]
    k = torch.where(s > 0, (v / torch.where(s > 0, s, 1.0)).float().double().round(), 0.0)
    return (k * s).view(-1)[:n]
