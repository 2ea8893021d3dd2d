"""Prompt and batch operators measured: cases, inputs, plain forms, 64-bit values.

Four operators take a prompt into the decode path of this library: rows of a
quantised embedding table, the norm and rotation of queries and keys, causal
attention over packed prompts, and one decode step's attention for a batch
whose sequences share a long prefix.  The plain forms are elementary torch
operations in f32; with ``own`` the library's entry points are called.
"""
import math

import torch

own = False

Q4_0, Q8_0, Q4_K, Q6_K = 2, 8, 12, 14
BLOCK = {Q4_0: (32, 18), Q8_0: (32, 34), Q4_K: (256, 144), Q6_K: (256, 210)}  # values, bytes


# ------------------------------------------------------------------- cases
def listed():
    gemma = dict(nq=8, nkv=4, hd=256)      # the benchmark's head layout
    ragged = "1,515,64,2,1300,129,37,256,777,63,1,900"
    return [
        # one decode step's input row from the tied 262144 x 2560 Q4_0 table
        dict(name="embed_q4_0_one", op="embed", fmt=Q4_0, vocab=262144, hidden=2560, n=1,
             scale=50.596443),
        # a long prompt's rows, Q6_K table (the usual type of a K-quantised file)
        dict(name="embed_q6_k_4001", op="embed", fmt=Q6_K, vocab=262144, hidden=2560, n=4001,
             scale=50.596443),
        # decode: one token's heads
        dict(name="qk_one", op="qk", n=1, rot=256, base=1e6, eps=1e-6, norm=True, far=1000,
             **gemma),
        # a prompt of 4096 tokens straight out of the fused QKV product
        dict(name="qk_4096", op="qk", n=4096, rot=256, base=1e6, eps=1e-6, norm=True, far=0,
             **gemma),
        # partial rotation far into a long context, no norm weights, odd token count
        dict(name="qk_partial_1037", op="qk", n=1037, nq=16, nkv=4, hd=128, rot=64, base=1e4,
             eps=1e-6, norm=False, far=130000),
        # a short chat prompt: latency
        dict(name="prompt_37", op="prompt", lens="37", ctx="", softcap=0.0, **gemma),
        # many requests of different lengths in one call
        dict(name="prompt_ragged", op="prompt", lens=ragged, ctx="", softcap=50.0, nq=16, nkv=4,
             hd=128),
        # a long prompt in one call
        dict(name="prompt_8192", op="prompt", lens="8192", ctx="", softcap=0.0, **gemma),
        # the last chunk of a long prompt that is fed in pieces
        dict(name="prompt_chunk", op="prompt", lens="512", ctx="8000", softcap=0.0, **gemma),
        # a few requests over a system prompt
        dict(name="prefix_4x777", op="prefix", prefix=777, ctx="1,130,0,64", softcap=0.0, nq=8,
             nkv=2, hd=64),
        # odd batch, ragged own parts, a mid-size document as the prefix
        dict(name="prefix_12x4099", op="prefix", prefix=4099,
             ctx="0,1000,37,512,1,64,777,300,129,2,900,15", softcap=50.0, nq=16, nkv=4, hd=128),
        # a large batch over a long shared document: 268 MB of shared keys and values
        dict(name="prefix_32x32768", op="prefix", prefix=32768,
             ctx=",".join(str(1 + 16 * i) for i in range(32)), softcap=0.0, **gemma),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _heads(rng):
    nkv = rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 2, 3, 4])
    return nkv * group, nkv, rng.choice([32, 64, 128, 256])


def draw(rng):
    op = rng.choice(["embed", "qk", "prompt", "prompt", "prefix", "prefix"])
    if op == "embed":
        fmt = rng.choice([Q4_0, Q8_0, Q4_K, Q6_K])
        bw = BLOCK[fmt][0]
        return dict(op=op, fmt=fmt, vocab=_log_int(rng, 500, 200000),
                    hidden=bw * max(1, _log_int(rng, 256, 2560) // bw), n=_log_int(rng, 1, 4000),
                    scale=rng.choice([1.0, round(rng.uniform(8.0, 64.0), 4)]))
    nq, nkv, hd = _heads(rng)
    if op == "qk":
        n = min(_log_int(rng, 1, 4000), 4096 * 12 * 256 // ((nq + nkv) * hd))
        return dict(op=op, n=max(1, n), nq=nq, nkv=nkv, hd=hd,
                    rot=rng.choice([hd, hd, hd // 2]), base=rng.choice([1e4, 5e5, 1e6]),
                    eps=1e-6, norm=rng.random() < 0.7, far=rng.choice([0, 1000, 130000, 1000003]))
    softcap = rng.choice([0.0, 0.0, 30.0, 50.0])
    if op == "prompt":
        s = _log_int(rng, 1, 12)
        top = min(_log_int(rng, 8, 4000), int(math.sqrt(8192 ** 2 * 8 / nq / s / 4)))
        lens = [max(1, int(top * rng.random())) for _ in range(s - 1)] + [top]
        rng.shuffle(lens)
        ctx = ""
        if rng.random() < 0.3:        # chunks: keys of earlier chunks before the call's own
            ctx = ",".join(str(n + int(rng.random() * top)) for n in lens)
        return dict(op=op, lens=",".join(map(str, lens)), ctx=ctx, softcap=softcap, nq=nq,
                    nkv=nkv, hd=hd)
    b = _log_int(rng, 1, 48)
    room = 32768 * 4 * 256 // (nkv * hd)
    prefix = min(_log_int(rng, 1, 40000), room // 2)
    longest = max(1, min(_log_int(rng, 1, 1000), room // 2 // b))
    return dict(op=op, prefix=prefix,
                ctx=",".join(str(int(rng.random() * (longest + 1))) for _ in range(b)),
                softcap=softcap, nq=nq, nkv=nkv, hd=hd)


def _ints(text):
    return [int(t) for t in text.split(",")]


def _spans(case):
    lens = _ints(case["lens"])
    ctx = _ints(case["ctx"]) if case["ctx"] else lens
    return lens, ctx


def _starts(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return at


# ------------------------------------------------------------------- inputs
def _table(fmt, vocab, hidden, g):
    """Blocks of random codes with scales in [0.001, 0.02), uint8 [vocab][row bytes]."""
    bw, bb = BLOCK[fmt]
    nb = hidden // bw
    W = torch.randint(0, 256, (vocab, nb, bb), dtype=torch.uint8, device="cuda", generator=g)
    n16, at = (2, 0) if fmt == Q4_K else (1, 208) if fmt == Q6_K else (1, 0)
    d = torch.rand((vocab, nb, n16), device="cuda", generator=g) * 0.019 + 0.001
    W[:, :, at:at + 2 * n16] = d.half().view(torch.uint8)
    return W.view(vocab, nb * bb)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, device="cuda", generator=g)

    s = dict(case)
    if case["op"] == "embed":
        s["W"] = _table(case["fmt"], case["vocab"], case["hidden"], g)
        s["tokens"] = torch.randint(0, case["vocab"], (case["n"],), device="cuda", generator=g)
        return s
    nq, nkv, hd = case["nq"], case["nkv"], case["hd"]
    if case["op"] == "qk":
        # the rows of the fused QKV product: queries, keys, values side by side
        qkv = normal(case["n"], nq + 2 * nkv, hd)
        s["q"], s["k"] = qkv[:, :nq], qkv[:, nq:nq + nkv]
        s["w_q"] = 1 + 0.1 * normal(hd) if case["norm"] else None
        s["w_k"] = 1 + 0.1 * normal(hd) if case["norm"] else None
        s["positions"] = case["far"] + torch.arange(case["n"], device="cuda")
    elif case["op"] == "prompt":
        lens, ctx = _spans(case)
        s["q"] = normal(sum(lens), nq, hd)
        s["k"], s["v"] = normal(sum(ctx), nkv, hd), normal(sum(ctx), nkv, hd)
        s["cu_q"], s["cu_k"] = _starts(lens), _starts(ctx)
        # the padded batch of the plain form: a row of s["at_*"] is a sequence
        dev = torch.device("cuda")
        nq_t, nk_t = torch.tensor(lens, device=dev), torch.tensor(ctx, device=dev)
        iq, ik = torch.arange(max(lens), device=dev), torch.arange(max(ctx), device=dev)
        s["at_q"] = torch.tensor(s["cu_q"][:-1], device=dev)[:, None] + torch.minimum(
            iq[None], nq_t[:, None] - 1)
        s["at_k"] = torch.tensor(s["cu_k"][:-1], device=dev)[:, None] + torch.minimum(
            ik[None], nk_t[:, None] - 1)
        # key j is visible to query i of a sequence iff j <= i + (keys - queries)
        s["seen"] = ik[None, None, :] <= iq[None, :, None] + (nk_t - nq_t)[:, None, None]
        s["seq"] = torch.repeat_interleave(torch.arange(len(lens), device=dev), nq_t)
        s["row"] = torch.arange(sum(lens), device=dev) - torch.tensor(
            s["cu_q"][:-1], device=dev)[s["seq"]]
    else:
        ctx = _ints(case["ctx"])
        b, longest = len(ctx), max(max(ctx), 1)
        s["n_ctx"] = ctx
        s["q"] = normal(b, nq, hd)
        s["kp"], s["vp"] = normal(nkv, case["prefix"], hd), normal(nkv, case["prefix"], hd)
        s["kc"], s["vc"] = normal(b, nkv, longest, hd), normal(b, nkv, longest, hd)
        s["seen"] = torch.arange(longest, device="cuda")[None] < torch.tensor(
            ctx, device="cuda")[:, None]
    return s


# ------------------------------------------------------------------- one pass
def run(s):
    if own:
        from quantized_weight_streaming_q4k_gb300 import ops
        if s["op"] == "embed":
            return ops.embed_tokens(s["fmt"], s["W"], s["tokens"], s["vocab"], s["hidden"],
                                    s["scale"])
        if s["op"] == "qk":
            return ops.qk_norm_rope(s["q"], s["k"], s["positions"], s["rot"], s["base"],
                                    w_q=s["w_q"], w_k=s["w_k"], eps=s["eps"])
        scale = s["hd"] ** -0.5
        if s["op"] == "prompt":
            return ops.prompt_attention(s["q"], s["k"], s["v"], s["cu_q"], scale, s["softcap"],
                                        cu_seqlens_k=s["cu_k"])
        return ops.prefix_attention(s["q"], s["kp"], s["vp"], s["prefix"], s["kc"], s["vc"],
                                    s["n_ctx"], scale, s["softcap"])
    return {"embed": _plain_embed, "qk": _plain_qk, "prompt": _plain_prompt,
            "prefix": _plain_prefix}[s["op"]](s)


def _half(b):
    return b.contiguous().view(torch.float16).float()


def _plain_embed(s):
    bw, bb = BLOCK[s["fmt"]]
    r = s["W"][s["tokens"]].view(s["n"], s["hidden"] // bw, bb)
    if s["fmt"] == Q4_0:
        q = torch.cat([r[..., 2:] & 15, r[..., 2:] >> 4], -1).float() - 8
        w = _half(r[..., :2]) * q
    elif s["fmt"] == Q8_0:
        w = _half(r[..., :2]) * r[..., 2:].contiguous().view(torch.int8).float()
    elif s["fmt"] == Q4_K:
        f = r[..., 4:16]
        sc = torch.cat([f[..., :4] & 63, (f[..., 8:] & 15) | ((f[..., :4] >> 6) << 4)], -1)
        mn = torch.cat([f[..., 4:8] & 63, (f[..., 8:] >> 4) | ((f[..., 4:8] >> 6) << 4)], -1)
        c = r[..., 16:].view(s["n"], -1, 4, 1, 32)
        q = torch.cat([c & 15, c >> 4], -2).view(s["n"], -1, 8, 32).float()
        w = (_half(r[..., :2]) * sc.float())[..., None] * q - (
            _half(r[..., 2:4]) * mn.float())[..., None]
    else:
        lo = r[..., :128].reshape(s["n"], -1, 2, 2, 32)
        hi = r[..., 128:192].reshape(s["n"], -1, 2, 1, 32)
        low = torch.cat([lo & 15, lo >> 4], -2)                      # [.., half, quarter, 32]
        top = torch.cat([hi & 3, (hi >> 2) & 3, (hi >> 4) & 3, hi >> 6], -2)
        q = (low | (top << 4)).reshape(s["n"], -1, 16, 16).float() - 32
        sc = r[..., 192:208].contiguous().view(torch.int8).float()
        w = (_half(r[..., 208:210]) * sc)[..., None] * q
    return w.reshape(s["n"], s["hidden"]) * s["scale"]


def _plain_qk(s):
    half = s["rot"] // 2
    i = torch.arange(half, device="cuda", dtype=torch.float64)
    # far positions: the angle in 64 bits
    theta = s["positions"].double()[:, None] * torch.pow(
        torch.tensor(s["base"], dtype=torch.float64, device="cuda"), -2 * i / s["rot"])
    c, sn = torch.cos(theta).float()[:, None], torch.sin(theta).float()[:, None]

    def one(x, w):
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * w
        a, b = x[..., :half], x[..., half:2 * half]
        return torch.cat([a * c - b * sn, a * sn + b * c, x[..., 2 * half:]], -1)

    return one(s["q"], s["w_q"]), one(s["k"], s["w_k"])


def _cap(x, cap):
    return cap * torch.tanh(x / cap) if cap > 0 else x


def _softmax_parts(x, seen):
    x = torch.where(seen, x, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
    l = p.sum(-1, keepdim=True)
    return p, torch.where(l == 0, 1.0, l)


def _plain_prompt(s):
    nq, nkv, hd = s["nq"], s["nkv"], s["hd"]
    n, lq = s["at_q"].shape
    lk, grp = s["at_k"].shape[1], nq // nkv
    q = s["q"][s["at_q"]].view(n, lq, nkv, grp, hd).permute(0, 2, 3, 1, 4)
    k = s["k"][s["at_k"]].permute(0, 2, 1, 3)
    v = s["v"][s["at_k"]].permute(0, 2, 1, 3)
    x = torch.matmul(q.reshape(n, nkv, grp * lq, hd) * hd ** -0.5, k.transpose(-1, -2))
    x = _cap(x.view(n, nkv, grp, lq, lk), s["softcap"])
    p, l = _softmax_parts(x, s["seen"][:, None, None])
    o = torch.matmul(p.view(n, nkv, grp * lq, lk), v).view(n, nkv, grp, lq, hd) / l
    return o.permute(0, 3, 1, 2, 4).reshape(n, lq, nq, hd)[s["seq"], s["row"]]


def _plain_prefix(s):
    nq, nkv, hd = s["nq"], s["nkv"], s["hd"]
    b, grp = s["q"].shape[0], nq // nkv
    q = s["q"].view(b, nkv, grp, hd) * hd ** -0.5
    # the shared part once for all rows of a head, the own parts row by row
    qh = q.transpose(0, 1).reshape(nkv, b * grp, hd)
    xp = torch.matmul(qh, s["kp"].transpose(-1, -2)).view(nkv, b, grp, -1).transpose(0, 1)
    xc = torch.matmul(q, s["kc"].transpose(-1, -2))
    x = _cap(torch.cat([xp, xc], -1), s["softcap"])
    n = s["prefix"]
    seen = torch.cat([torch.ones_like(s["seen"][:, :1]).expand(b, n), s["seen"]], 1)
    p, l = _softmax_parts(x, seen[:, None, None])
    ph = p[..., :n].transpose(0, 1).reshape(nkv, b * grp, n)
    o = torch.matmul(ph, s["vp"]).view(nkv, b, grp, hd).transpose(0, 1)
    o = (o + torch.matmul(p[..., n:], s["vc"])) / l
    return o.reshape(b, nq, hd)


# ------------------------------------------------------------------- what a pass needs
def work(case):
    if case["op"] == "embed":
        bw, bb = BLOCK[case["fmt"]]
        n, h = case["n"], case["hidden"]
        return {"bytes": n * (h // bw * bb + 4 * h + 8), "flops": 3 * n * h}
    nq, nkv, hd = case["nq"], case["nkv"], case["hd"]
    if case["op"] == "qk":
        vals = case["n"] * (nq + nkv) * hd
        return {"bytes": 8 * vals + 8 * case["n"] + (8 * hd if case["norm"] else 0),
                "flops": 8 * vals}
    if case["op"] == "prompt":
        lens, ctx = _spans(case)
        pairs = sum(n * c - n * (n - 1) // 2 for n, c in zip(lens, ctx))
        return {"bytes": 8 * hd * (nq * sum(lens) + nkv * sum(ctx)),
                "flops": 4 * pairs * nq * hd}
    ctx = _ints(case["ctx"])
    keys = case["prefix"] + sum(ctx)
    pairs = len(ctx) * case["prefix"] + sum(ctx)
    return {"bytes": 8 * hd * (nq * len(ctx) + nkv * keys), "flops": 4 * pairs * nq * hd}


# ------------------------------------------------------------------- 64-bit values
def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "embed":
        return _exact_embed(s)
    if s["op"] == "qk":
        return _exact_qk(s)
    if s["op"] == "prompt":
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        for a, b, c, d in zip(s["cu_q"], s["cu_q"][1:], s["cu_k"], s["cu_k"][1:]):
            for h in range(s["nq"]):
                g = h * s["nkv"] // s["nq"]
                for r in range(a, b, 2048):          # rows in pieces: memory
                    e = min(b, r + 2048)
                    last = torch.arange(r - a, e - a, device="cuda") + (d - c) - (b - a)
                    out[r:e, h] = _exact_rows(s["q"][r:e, h], s["k"][c:d, g], s["v"][c:d, g],
                                              last, s)
        return out
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for g in range(s["nkv"]):
        grp = s["nq"] // s["nkv"]
        for b, n in enumerate(s["n_ctx"]):
            k = torch.cat([s["kp"][g], s["kc"][b, g, :n]])
            v = torch.cat([s["vp"][g], s["vc"][b, g, :n]])
            last = torch.full((grp,), k.shape[0], device="cuda")
            out[b, g * grp:(g + 1) * grp] = _exact_rows(s["q"][b, g * grp:(g + 1) * grp], k, v,
                                                        last, s)
    return out


def _exact_rows(q, k, v, last, s):
    """Rows q over keys 0 .. last[row], from the definition, in f64."""
    z = torch.einsum("id,jd->ij", q.double(), k.double()) / math.sqrt(s["hd"])
    if s["softcap"]:
        z = torch.tanh(z / s["softcap"]) * s["softcap"]
    z = z.masked_fill(torch.arange(k.shape[0], device="cuda")[None] > last[:, None], -math.inf)
    return torch.einsum("ij,jd->id", torch.softmax(z, 1).nan_to_num(0.0), v.double())


def _exact_qk(s):
    def one(x, w):
        y = x.double().clone()
        if w is not None:
            y = y / torch.sqrt((y ** 2).sum(-1, keepdim=True) / y.shape[-1] + s["eps"])
            y = y * w.double()
        r = s["rot"]
        freq = [math.pow(s["base"], -2.0 * i / r) for i in range(r // 2)]
        ang = torch.outer(s["positions"].double(),
                          torch.tensor(freq, dtype=torch.float64, device="cuda"))
        z = torch.complex(y[..., :r // 2], y[..., r // 2:r]) * torch.polar(
            torch.ones_like(ang), ang)[:, None]
        y[..., :r // 2], y[..., r // 2:r] = z.real, z.imag
        return y

    return one(s["q"], s["w_q"]), one(s["k"], s["w_k"])


def _exact_embed(s):
    """Value by value from the block layouts: column c of a block."""
    fmt = s["fmt"]
    bw, bb = BLOCK[fmt]
    blocks = s["W"].view(s["vocab"], -1, bb)[s["tokens"]].to(torch.int32)     # [n, nb, bytes]

    def f16(at):
        u = (blocks[..., at] | (blocks[..., at + 1] << 8)).to(torch.int32)
        e, m = (u >> 10) & 31, (u & 1023).double()
        val = torch.where(e == 0, m * 2.0 ** -24, (1 + m / 1024) * torch.pow(2.0, e.double() - 15))
        return torch.where(u >= 32768, -val, val)

    def i8(b):
        return torch.where(b > 127, b - 256, b).double()

    c = torch.arange(bw, device="cuda")
    if fmt == Q4_0:
        code = (blocks[..., 2 + c % 16] >> (4 * (c // 16))) & 15
        w = f16(0)[..., None] * (code.double() - 8)
    elif fmt == Q8_0:
        w = f16(0)[..., None] * i8(blocks[..., 2 + c])
    elif fmt == Q4_K:
        j = c // 32                                                           # sub-block
        code = (blocks[..., 16 + 32 * (c // 64) + c % 32] >> (4 * (j % 2))) & 15
        jj = j % 4
        lo_s, lo_m, both = blocks[..., 4 + jj], blocks[..., 8 + jj], blocks[..., 12 + jj]
        first = j < 4
        sc = torch.where(first, lo_s % 64, both % 16 + 16 * (lo_s // 64))
        mn = torch.where(first, lo_m % 64, both // 16 + 16 * (lo_m // 64))
        w = f16(0)[..., None] * sc.double() * code.double() - f16(2)[..., None] * mn.double()
    else:
        h, r = c // 128, c % 128                                              # half, place in it
        quarter, l = r // 32, r % 32
        low = (blocks[..., 64 * h + 32 * (quarter % 2) + l] >> (4 * (quarter // 2))) & 15
        top = (blocks[..., 128 + 32 * h + l] >> (2 * quarter)) & 3
        w = f16(208)[..., None] * i8(blocks[..., 192 + c // 16]) * (low + 16 * top - 32).double()
    return w.reshape(s["n"], s["hidden"]) * float(s["scale"])
