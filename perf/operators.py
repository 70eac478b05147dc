"""Cases of the operators at the two ends of the data-parallel step, each in a
plain form (elementary torch operations) and as calls of libzq:

sumsq   the sum of squares over many gradient tensors (binary64)
clip    the global norm and the gradients scaled by min(1, max_norm / (norm + eps))
lookup  embedding rows times a scale, from a table or from its qwZ int8 codes
grad    the table's gradient from the tokens' gradients: written, added (fp32),
        or added with stochastic rounding (bf16)

Table sizes are those of the repository's models (vocabularies 32000 and
50257; widths 768, 2048, 4096) or generic.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
BYTES = {"fp32": 4, "bf16": 2, "fp16": 2}
EPS = 1e-6
M32 = 0xFFFFFFFF


def listed():
    return [
        # A small model's gradients: the call is launches and latency.
        {"name": "norm_small_fp32", "op": "sumsq", "type": "fp32", "layers": 2, "width": 256, "ffn": 688, "vocab": 1000,
         "odd": 0},
        # The ~0.85B model's 129 gradients in bf16: what a rank sums before the scalar all-reduce.
        {"name": "norm_0.85B_bf16", "op": "sumsq", "type": "bf16", "layers": 14, "width": 2048, "ffn": 5632,
         "vocab": 32000, "odd": 0},
        # A 124M-parameter model's tensors with ragged sizes, bf16: every tensor ends inside a tile.
        {"name": "clip_124M_bf16_ragged", "op": "clip", "type": "bf16", "layers": 12, "width": 768, "ffn": 2048,
         "vocab": 50257, "odd": 1, "max_norm": 1.0},
        # The same model's 8-way shard in fp16: 111 pieces, a call of tens of microseconds.
        {"name": "clip_shard_fp16", "op": "clip", "type": "fp16", "layers": 12, "width": 272, "ffn": 720,
         "vocab": 6283, "odd": 1, "max_norm": 1.0},
        # The ~0.85B model's reduced fp32 gradients: the largest.
        {"name": "clip_0.85B_fp32", "op": "clip", "type": "fp32", "layers": 14, "width": 2048, "ffn": 5632,
         "vocab": 32000, "odd": 0, "max_norm": 1.0},
        # One token, as in decoding.
        {"name": "lookup_1_token_bf16", "op": "lookup", "table": "bf16", "out": "bf16", "rows": 32000, "dim": 4096,
         "tokens": 1, "block": 0, "long": True, "pad": 0},
        # A micro-batch of 8 x 1024 tokens on the 124M model's fp32 table, int32 ids, padded sequences.
        {"name": "lookup_8192_fp32_bf16", "op": "lookup", "table": "fp32", "out": "bf16", "rows": 50257, "dim": 768,
         "tokens": 8192, "block": 0, "long": False, "pad": 10},
        # The 7.5B model's rows straight from what the qwZ all-gather delivered (int8, block 2048).
        {"name": "lookup_16384_int8_bf16", "op": "lookup", "table": "int8", "out": "bf16", "rows": 32000, "dim": 4096,
         "tokens": 16384, "block": 2048, "long": True, "pad": 0},
        # Few tokens, an odd width, a small vocabulary.
        {"name": "grad_write_odd_fp16", "op": "grad", "mode": "write", "dout": "fp16", "grad": "fp16", "rows": 1000,
         "dim": 1001, "tokens": 65, "long": False, "pad": 5},
        # The 124M model's bf16 accumulator, a micro-batch of 8 x 1024 tokens, stochastic rounding.
        {"name": "grad_sr_8192_bf16", "op": "grad", "mode": "add_sr", "dout": "bf16", "grad": "bf16", "rows": 50257,
         "dim": 768, "tokens": 8192, "long": False, "pad": 0},
        # The ~0.85B model: the first micro-batch writes the fp32 gradient of the whole table.
        {"name": "grad_write_16384_fp32", "op": "grad", "mode": "write", "dout": "bf16", "grad": "fp32", "rows": 32000,
         "dim": 2048, "tokens": 16384, "long": True, "pad": 10},
        # The 7.5B model: later micro-batches add into it.
        {"name": "grad_add_32768_fp32", "op": "grad", "mode": "add", "dout": "bf16", "grad": "fp32", "rows": 32000,
         "dim": 4096, "tokens": 32768, "long": True, "pad": 0},
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["sumsq", "clip", "lookup", "grad"])
    if op in ("sumsq", "clip"):
        c = {"op": op, "type": rng.choice(sorted(TYPES)), "layers": spread(1, 14), "width": spread(64, 2048),
             "ffn": spread(64, 5632), "vocab": spread(100, 32000), "odd": rng.randrange(2)}
        if op == "clip":
            c["max_norm"] = rng.choice([0.1, 1.0, 1e9])
        return c
    c = {"op": op, "rows": spread(50, 50257), "dim": spread(16, 4096), "tokens": spread(1, 32768),
         "long": rng.random() < 0.5, "pad": rng.choice([0, 10])}
    while c["rows"] * c["dim"] > 32000 * 4096 or c["tokens"] * c["dim"] > 1 << 26:
        c["dim"] = max(16, c["dim"] // 2)
    if op == "lookup":
        c["table"] = rng.choice(["int8"] + sorted(TYPES))
        c["block"] = 1 << rng.randrange(5, 13) if c["table"] == "int8" else 0
        c["out"] = rng.choice(sorted(TYPES))
    else:
        c["mode"] = rng.choice(["write", "write", "add", "add_sr"])
        c["dout"] = rng.choice(sorted(TYPES))
        c["grad"] = {"add": "fp32", "add_sr": "bf16"}.get(c["mode"]) or rng.choice(sorted(TYPES))
    return c


def sizes(case):
    """A Llama-style model's tensors; with `odd` each is some elements longer."""
    h, f, v = case["width"], case["ffn"], case["vocab"]
    n = [v * h] + case["layers"] * [h, h * h, h * h, h * h, h * h, h, f * h, f * h, h * f] + [h, v * h]
    return [x + (1 + 37 * i % 61 if case["odd"] else 0) for i, x in enumerate(n)]


def views(flat, numels):
    """The tensors in a flat buffer, each on a 64-element boundary."""
    out, at = [], 0
    for n in numels:
        out.append(flat[at:at + n])
        at += -(-n // 64) * 64
    return out


def flat_len(numels):
    return sum(-(-n // 64) * 64 for n in numels)


def generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def draw_ids(case, gen):
    """Token ids as text has them: log-uniform ranks (a Zipf law), spread over
    the vocabulary; `pad` % of the tokens are padding (-1)."""
    rows, n = case["rows"], case["tokens"]
    u = torch.rand(n, generator=gen, device="cuda", dtype=torch.float64)
    rank = ((rows + 1.0) ** u).long().sub_(1).clamp_(0, rows - 1)
    ids = (rank * 7919 + 13) % rows
    if case["pad"]:
        ids = torch.where(torch.rand(n, generator=gen, device="cuda") * 100 < case["pad"], -1, ids)
    return ids if case["long"] else ids.int()


def prepare(case, seed):
    gen = generator(seed)
    s = dict(case)
    if case["op"] in ("sumsq", "clip"):
        n, t = sizes(case), TYPES[case["type"]]
        flat = torch.empty(flat_len(n), device="cuda", dtype=t)
        for i in range(0, flat.numel(), 1 << 28):
            part = flat[i:i + (1 << 28)]
            part.copy_(torch.randn(part.numel(), generator=gen, device="cuda").mul_(1e-3))
        s["grads"] = views(flat, n)
        if case["op"] == "clip":
            s["flat_out"] = torch.zeros(flat.numel(), device="cuda", dtype=t)
            s["outs"] = views(s["flat_out"], n)
        if own:  # the table and workspace that a training program keeps beside its buffers
            from weight_communication_zero_amd import zq
            s["segments"] = zq.GradSegmentTable(zip(s["grads"], s.get("outs") or s["grads"]))
            s["sumsq"] = torch.empty(1, device="cuda", dtype=torch.float64)
            s["norm"] = torch.empty(1, device="cuda")
            s["workspace"] = torch.empty(zq.grad_sumsq_workspace(len(n)), device="cuda", dtype=torch.uint8)
        return s
    rows, dim, n = case["rows"], case["dim"], case["tokens"]
    s["ids"] = draw_ids(case, gen)
    s["scale"] = math.sqrt(dim)
    if case["op"] == "lookup":
        if case["table"] == "int8":
            b = case["block"]
            s["codes"] = torch.randint(-127, 128, (rows, dim), generator=gen, device="cuda", dtype=torch.int8)
            s["scales"] = torch.rand(-(-rows * dim // b), generator=gen, device="cuda").add_(0.5).mul_(4e-4)
        else:
            s["weight"] = torch.randn(rows, dim, generator=gen, device="cuda").mul_(0.02).to(TYPES[case["table"]])
        s["result"] = torch.empty(n, dim, device="cuda", dtype=TYPES[case["out"]])
        return s
    s["dy"] = torch.randn(n, dim, generator=gen, device="cuda").mul_(1e-4).to(TYPES[case["dout"]])
    s["dw"] = torch.randn(rows, dim, generator=gen, device="cuda").mul_(1e-4).to(TYPES[case["grad"]])
    s["seed"], s["base"] = (seed * 0x9E3779B97F4A7C15 + 1) & 0x7FFFFFFFFFFFFFFF, 8 * (seed % 1000) + seed % 8
    if own:
        from weight_communication_zero_amd import zq
        s["workspace"] = torch.empty(zq.embed_grad_workspace(n, rows, dim), device="cuda", dtype=torch.uint8)
    return s


def run(s):
    if own:
        return run_own(s)
    if s["op"] in ("sumsq", "clip"):
        q = torch.stack([g.double().square().sum() for g in s["grads"]]).sum()
        if s["op"] == "sumsq":
            return {"sumsq": q.reshape(1)}
        norm = q.sqrt()
        c = (s["max_norm"] / (norm + EPS)).clamp(max=1.0).float()
        torch._foreach_copy_(s["outs"], [(g.float() * c).to(g.dtype) for g in s["grads"]])
        return {"norm": norm.float().reshape(1), "out": s["flat_out"]}
    ids = s["ids"].long()
    there = (ids >= 0) & (ids < s["rows"])
    if s["op"] == "lookup":
        at = torch.where(there, ids, 0)
        if s["table"] == "int8":
            e = at[:, None] * s["dim"] + torch.arange(s["dim"], device="cuda")
            w = s["codes"][at].float() * s["scales"][e // s["block"]]
        else:
            w = s["weight"][at].float()
        return {"out": torch.where(there[:, None], w * s["scale"], 0.0).to(s["result"].dtype)}
    dw, at = s["dw"], ids[there]
    g = s["dy"][there].float() * s["scale"]
    if s["mode"] == "write":
        dw.copy_(torch.zeros(dw.shape, device="cuda").index_add_(0, at, g))
    elif s["mode"] == "add":
        dw.index_add_(0, at, g)
    else:
        named = torch.zeros(s["rows"], device="cuda", dtype=torch.bool).index_fill_(0, at, True)
        x = torch.zeros(dw.shape, device="cuda").index_add_(0, at, g).add_(dw)
        bits = (x.view(torch.int32).long() & M32) + random16(s["seed"], s["base"], dw.numel()).reshape(dw.shape)
        bits = torch.where(x.isnan(), 0x7FC0, (bits & M32) >> 16)
        new = torch.where(bits >= 1 << 15, bits - (1 << 16), bits).to(torch.int16).view(torch.bfloat16)
        dw.copy_(torch.where(named[:, None], new, dw))
    return {"grad": dw}


def random16(seed, base, n):
    """The 16-bit numbers of elements base .. base + n - 1: Philox4x32-10 of
    counter q >> 3 with the seed as key, eight numbers from each call."""
    first, last = base >> 3, (base + n + 7) >> 3
    c = torch.arange(first, last, device="cuda")
    zero = torch.zeros_like(c)
    w, key = (c & M32, c >> 32, zero, zero), (seed & M32, seed >> 32)
    for _ in range(10):
        h0, l0 = product(0xD2511F53, w[0])
        h1, l1 = product(0xCD9E8D57, w[2])
        w = (h1 ^ w[1] ^ key[0], l1, h0 ^ w[3] ^ key[1], l0)
        key = ((key[0] + 0x9E3779B9) & M32, (key[1] + 0xBB67AE85) & M32)
    halves = torch.stack([h for x in w for h in (x & 0xFFFF, x >> 16)], dim=1).reshape(-1)
    return halves[base - 8 * first:][:n]


def product(m, x):
    """The high and low words of a 32 x 32 bit product."""
    lo, hi = x * (m & 0xFFFF), x * (m >> 16)
    return (hi + (lo >> 16)) >> 16, (lo + ((hi & 0xFFFF) << 16)) & M32


def run_own(s):
    from weight_communication_zero_amd import zq
    if s["op"] in ("sumsq", "clip"):
        zq.zq_grad_sumsq_batched(s["segments"], s["sumsq"], s["workspace"])
        if s["op"] == "sumsq":
            return {"sumsq": s["sumsq"]}
        zq.zq_grad_clip_batched(s["segments"], s["sumsq"], s["max_norm"], EPS, norm=s["norm"])
        return {"norm": s["norm"], "out": s["flat_out"]}
    if s["op"] == "lookup":
        if s["table"] == "int8":
            zq.zq_embed_lookup_int8(s["codes"], s["scales"], s["block"], s["ids"], s["scale"], s["result"])
        else:
            zq.zq_embed_lookup(s["weight"], s["ids"], s["scale"], s["result"])
        return {"out": s["result"]}
    mode = {"write": zq.ZQ_GRAD_WRITE, "add": zq.ZQ_GRAD_ADD, "add_sr": zq.ZQ_GRAD_ADD_SR}[s["mode"]]
    zq.zq_embed_grad(s["dy"], s["ids"], s["scale"], s["dw"], mode, s["workspace"], seed=s["seed"],
                     counter_base=s["base"])
    return {"grad": s["dw"]}


def distinct(case):
    """Expected number of distinct rows that the tokens name."""
    rows, n = case["rows"], case["tokens"] * (1 - case["pad"] / 100)
    r = np.arange(rows, dtype=np.float64)
    p = np.log((r + 2) / (r + 1)) / math.log(rows + 1)
    return float((1 - (1 - p) ** n).sum())


def work(case):
    if case["op"] in ("sumsq", "clip"):
        n, b = sum(sizes(case)), BYTES[case["type"]]
        return {"bytes": n * b + 8 if case["op"] == "sumsq" else 2 * n * b + 4,
                "flops": 2 * n if case["op"] == "sumsq" else 3 * n}
    n, d, rows = case["tokens"], case["dim"], case["rows"]
    ids = n * (8 if case["long"] else 4)
    if case["op"] == "lookup":
        b = 1 + 4 / case["block"] if case["table"] == "int8" else BYTES[case["table"]]
        return {"bytes": ids + distinct(case) * d * b + n * d * BYTES[case["out"]],
                "flops": n * d * (2 if case["table"] == "int8" else 1)}
    valid = n * (1 - case["pad"] / 100)
    g = BYTES[case["grad"]] * d * (rows if case["mode"] == "write" else 2 * distinct(case))
    return {"bytes": ids + valid * d * BYTES[case["dout"]] + g, "flops": valid * d + distinct(case) * d}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("sumsq", "clip"):
        parts = [p.double() for g in s["grads"] for p in g.split(1 << 24)]
        q = math.fsum(float(torch.dot(p, p)) for p in parts)
        if case["op"] == "sumsq":
            return {"sumsq": np.array([q])}
        c = min(1.0, case["max_norm"] / (math.sqrt(q) + EPS))
        out = torch.zeros(s["flat_out"].numel(), device="cuda", dtype=torch.float64)
        for o, g in zip(views(out, sizes(case)), s["grads"]):
            o.copy_(g).mul_(c)
        return {"norm": np.array([math.sqrt(q)]), "out": out}
    ids = s["ids"].cpu().long().numpy()
    there = (ids >= 0) & (ids < case["rows"])
    if case["op"] == "lookup":
        out = torch.zeros(s["result"].shape, device="cuda", dtype=torch.float64)
        t, i = (torch.from_numpy(x).cuda() for x in (np.nonzero(there)[0], ids[there]))
        if case["table"] == "int8":
            blocks = s["scales"].double().repeat_interleave(case["block"])[:s["codes"].numel()]
            w = (s["codes"].double().reshape(-1) * blocks).reshape(s["codes"].shape)
        else:
            w = s["weight"].double()
        out[t] = w[i] * s["scale"]
        return {"out": out}
    order = np.nonzero(there)[0][np.argsort(ids[there], kind="stable")]
    named, first = np.unique(ids[order], return_index=True)
    total = torch.zeros(len(order) + 1, case["dim"], device="cuda", dtype=torch.float64)
    torch.cumsum(s["dy"][torch.from_numpy(order).cuda()].double(), 0, out=total[1:])
    edges = torch.from_numpy(np.append(first, len(order))).cuda()
    g = (total[edges[1:]] - total[edges[:-1]]) * s["scale"]
    old, at = s["dw"].double(), torch.from_numpy(named).cuda()
    if case["mode"] == "write":
        old.zero_()
    old[at] += g
    if case["mode"] != "add_sr":
        return {"grad": old}
    x = old[at].float().cpu().numpy().view(np.uint32).astype(np.uint64)
    q = (named[:, None] * case["dim"] + np.arange(case["dim"]) + s["base"]).astype(np.uint64)
    new = ((x + exact_random16(s["seed"], q)) & np.uint64(M32)) >> np.uint64(16)
    old[at] = torch.from_numpy((new << np.uint64(16)).astype(np.uint32).view(np.float32)).cuda().double()
    return {"grad": old}


def exact_random16(seed, q):
    """The 16-bit numbers of the elements q, one Philox4x32-10 call for each."""
    u, m = np.uint64, np.uint64(M32)
    x0, x1, x2, x3 = (q >> u(3)) & m, q >> u(35), np.zeros_like(q), np.zeros_like(q)
    k0, k1 = u(seed & M32), u(seed >> 32)
    for i in range(10):
        a, b = x0 * u(0xD2511F53), x2 * u(0xCD9E8D57)
        x0, x1, x2, x3 = (b >> u(32)) ^ x1 ^ k0, b & m, (a >> u(32)) ^ x3 ^ k1, a & m
        k0, k1 = (k0 + u(0x9E3779B9)) & m, (k1 + u(0xBB67AE85)) & m
    word = np.choose(((q & u(7)) >> u(1)).astype(np.int64), [x0, x1, x2, x3])
    return np.where(q & u(1), word >> u(16), word & u(0xFFFF))
