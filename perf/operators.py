"""The attention operators, as cases to be measured: appending normed and rotated keys and values to a paged
cache, attention over packed prompts, and attention of single tokens over a paged cache with a shared prefix.

``run`` computes an operator either in its plain form (elementary torch operations in 32 bits, rounded once at the
end) or, with ``own``, through the library's entry points.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # one new token of one sequence: the smallest call of a decode step, where latency counts
        dict(name="append 1 token", op="append", T=1, Hq=32, Hkv=4, D=128, rot=128, interleaved=False, norm=True,
             page=16, prompt=False, max_pos=40960, dtype="bf16"),
        # one token for each of 256 sequences of a decode batch
        dict(name="append 256 tokens", op="append", T=256, Hq=32, Hkv=4, D=128, rot=128, interleaved=False, norm=True,
             page=16, prompt=False, max_pos=40960, dtype="bf16"),
        # a prompt of an odd length on a small-head model: interleaved pairs on half of the head, no norms
        dict(name="append 1021 interleaved f16", op="append", T=1021, Hq=12, Hkv=3, D=64, rot=32, interleaved=True,
             norm=False, page=64, prompt=True, max_pos=4096, dtype="f16"),
        # a whole prefill chunk
        dict(name="append 8192 prompt", op="append", T=8192, Hq=32, Hkv=4, D=128, rot=128, interleaved=False,
             norm=True, page=16, prompt=True, max_pos=16384, dtype="bf16"),
        # many short prompts of different lengths in one batch, a few of a single token
        dict(name="prefill 37 ragged", op="prefill", n=37, q_low=1, q_high=700, hist=0, Hq=32, Hkv=4, D=128,
             causal=True, page=0, lse=False, dtype="bf16", shape_seed=1),
        # sequences of a bidirectional encoder: every head has keys of its own, no causal mask
        dict(name="prefill 16 full f16", op="prefill", n=16, q_low=100, q_high=1000, hist=0, Hq=12, Hkv=12, D=64,
             causal=False, page=0, lse=False, dtype="f16", shape_seed=2),
        # chunks of long prompts: new tokens read the history of their sequence from the paged cache
        dict(name="prefill 4 chunks paged", op="prefill", n=4, q_low=300, q_high=1024, hist=7000, Hq=32, Hkv=4, D=128,
             causal=True, page=16, lse=True, dtype="bf16", shape_seed=3),
        # one prompt as long as a prefill chunk
        dict(name="prefill 8192", op="prefill", n=1, q_low=8192, q_high=8192, hist=0, Hq=32, Hkv=4, D=128,
             causal=True, page=0, lse=False, dtype="bf16", shape_seed=4),
        # a small decode batch over short contexts: latency counts
        dict(name="decode 8 short f16", op="decode", B=8, kv_low=100, kv_high=700, prefix=0, Hq=16, Hkv=2, D=64,
             page=16, lse=False, dtype="f16", shape_seed=5),
        # an ordinary decode batch of very different lengths
        dict(name="decode 64 ragged", op="decode", B=64, kv_low=1, kv_high=8192, prefix=0, Hq=32, Hkv=4, D=128,
             page=16, lse=False, dtype="bf16", shape_seed=6),
        # one sequence with a very long context: few rows, a long axis
        dict(name="decode 1 long", op="decode", B=1, kv_low=131001, kv_high=131001, prefix=0, Hq=32, Hkv=4, D=128,
             page=64, lse=False, dtype="bf16", shape_seed=7),
        # requests that share a long system prompt or document
        dict(name="decode 64 shared 16k", op="decode", B=64, kv_low=50, kv_high=700, prefix=16384, Hq=32, Hkv=4,
             D=128, page=16, lse=True, dtype="bf16", shape_seed=8),
    ]


def _log(rng, low, high):
    """A whole number between low and high, spread over the logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["append", "prefill", "prefill", "decode", "decode"])
    D = rng.choice([64, 128])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 4, 6, 7, 8])
    if Hq > 32:
        Hq = Hkv * 4
    if op == "append":
        return dict(op=op, T=_log(rng, 1, 8192), Hq=Hq, Hkv=Hkv, D=D, rot=rng.choice([16, 32, 64, D, D]),
                    interleaved=rng.random() < 0.4, norm=rng.random() < 0.6, page=rng.choice([16, 32, 64, 128]),
                    prompt=rng.random() < 0.5, max_pos=rng.choice([8192, 16384, 40960]), dtype=dtype)
    shape_seed = rng.randrange(1 << 20)
    if op == "prefill":
        n = _log(rng, 1, 64)
        page = rng.choice([0, 0, 16, 32, 64, 128])
        q_high = _log(rng, 2, int(8192 / math.sqrt(n)))
        # n * q_high * (q_high + hist) stays within one prompt of 8192 tokens
        hist = rng.randrange(0, max(1, min(8192, 8192 * 8192 // (2 * n * q_high) - q_high))) if page else 0
        return dict(op=op, n=n, q_low=max(1, q_high // rng.choice([1, 3, 50])), q_high=q_high, hist=hist, Hq=Hq, Hkv=Hkv,
                    D=D, causal=rng.random() < 0.8, page=page, lse=rng.random() < 0.3, dtype=dtype,
                    shape_seed=shape_seed)
    B = _log(rng, 1, 256)
    # B * kv_high * Hkv * D stays within one long context of the listed case
    kv_high = _log(rng, 16, max(16, min(131072, 131072 * 512 // (B * Hkv * D))))
    prefix = rng.choice([0, 0, _log(rng, 100, 16384)])
    return dict(op=op, B=B, kv_low=max(1, kv_high // rng.choice([1, 4, 100])), kv_high=kv_high, prefix=prefix, Hq=Hq,
                Hkv=Hkv, D=D, page=rng.choice([16, 32, 64, 128]), lse=rng.random() < 0.3, dtype=dtype,
                shape_seed=shape_seed)


def _lengths(case):
    """Lengths of a case's sequences: (query tokens, keys) for each."""
    r = random.Random(case["shape_seed"])
    if case["op"] == "decode":
        return [(1, _log(r, case["kv_low"], case["kv_high"])) for _ in range(case["B"])]
    q = [_log(r, case["q_low"], case["q_high"]) for _ in range(case["n"])]
    return [(a, a + (r.randint(case["hist"] // 4, case["hist"]) if case["hist"] else 0)) for a in q]


def _starts(lens):
    s = [0]
    for v in lens:
        s.append(s[-1] + v)
    return s


def _ints(values, device="cuda"):
    return torch.tensor(values, dtype=torch.int32, device=device)


def _pages(lens, page, gen):
    """Page lists of sequences of these lengths, scattered over a pool with a few spare pages: (table, pool size)."""
    need = [(v + page - 1) // page for v in lens]
    pool = sum(need) + 3
    order = torch.randperm(pool, generator=gen, device="cuda").to(torch.int32)
    wide = max(1, max(need))
    at = torch.tensor(_starts(need)[:-1], device="cuda")[:, None] + torch.arange(wide, device="cuda")[None, :]
    used = torch.arange(wide, device="cuda")[None, :] < torch.tensor(need, device="cuda")[:, None]
    return torch.where(used, order[at.clamp(max=pool - 1)], 0).contiguous(), pool


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]

    def rand(*shape, mul=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * mul).to(dt)

    s = dict(case=case, ws=None, scale=1.0 / math.sqrt(D))
    if case["op"] == "append":
        T, page, rot = case["T"], case["page"], case["rot"]
        # q, k and v are parts of one projection's rows
        qkv = rand(T, (Hq + 2 * Hkv) * D, mul=2.0)
        s["q"] = qkv[:, :Hq * D].view(T, Hq, D)
        s["k"] = qkv[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D)
        s["v"] = qkv[:, (Hq + Hkv) * D:].view(T, Hkv, D)
        s["q_norm"] = s["k_norm"] = None
        if case["norm"]:
            s["q_norm"] = 1.0 + 0.3 * torch.randn(D, generator=gen, device="cuda")
            s["k_norm"] = 1.0 + 0.3 * torch.randn(D, generator=gen, device="cuda")
        inv = 1000000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
        angle = torch.arange(case["max_pos"], dtype=torch.float64, device="cuda")[:, None] * inv[None, :]
        s["table"] = torch.cat([angle.cos(), angle.sin()], dim=1).float().contiguous()
        pages = (T + page - 1) // page + 3
        order = torch.randperm(pages, generator=gen, device="cuda")
        if case["prompt"]:
            first = seed % 100 % (case["max_pos"] - T) if case["max_pos"] > T else 0
            s["positions"] = (torch.arange(T, device="cuda") + first).to(torch.int32)
            t = torch.arange(T, device="cuda")
            s["slots"] = (order[t // page] * page + t % page).to(torch.int32)
        else:
            s["positions"] = torch.randint(0, case["max_pos"], (T,), generator=gen, device="cuda", dtype=torch.int32)
            s["slots"] = torch.randperm(pages * page, generator=gen, device="cuda")[:T].to(torch.int32)
        s["k_cache"] = rand(pages, Hkv, page, D)
        s["v_cache"] = rand(pages, Hkv, page, D)
        s["q_out"] = torch.empty(T, Hq, D, dtype=dt, device="cuda")
    else:
        lens = _lengths(case)
        kv = [b for _, b in lens]
        rows = sum(a for a, _ in lens)
        s["q"] = rand(rows, Hq, D, mul=2.5)
        s["out"] = torch.empty(rows, Hq, D, dtype=dt, device="cuda")
        s["lse"] = torch.empty(rows, Hq, dtype=torch.float32, device="cuda") if case["lse"] else None
        s["max_q"], s["max_kv"] = max(a for a, _ in lens), max(kv)
        s["q_starts"] = _ints(_starts([a for a, _ in lens]))
        s["kv_lens"] = _ints(kv)
        if case["page"]:
            s["page_table"], pool = _pages(kv, case["page"], gen)
            prefix = case.get("prefix", 0)
            if prefix:
                n = (prefix + case["page"] - 1) // case["page"]
                s["prefix_table"] = (torch.randperm(n, generator=gen, device="cuda") + pool).to(torch.int32)
                pool += n
            s["k_cache"] = rand(pool, Hkv, case["page"], D)
            s["v_cache"] = rand(pool, Hkv, case["page"], D)
        else:
            s["kv_starts"] = _ints(_starts(kv))
            s["k"], s["v"] = rand(sum(kv), Hkv, D), rand(sum(kv), Hkv, D)
    if own:
        import expert_layer_gb300 as moe
        rows = case["T"] if case["op"] == "append" else s["q"].shape[0]
        s["ws"] = moe.alloc_attn_workspace(rows, case.get("n") or case.get("B") or 1, Hq, Hkv, D)
    return s


def run(s):
    op = s["case"]["op"]
    if own:
        return {"append": _own_append, "prefill": _own_prefill, "decode": _own_decode}[op](s)
    return {"append": _plain_append, "prefill": _plain_prefill, "decode": _plain_decode}[op](s)


# ------------------------------------------------------------------ the library
def _own_append(s):
    import expert_layer_gb300 as moe
    moe.rope_append(s["q"], s["k"], s["v"], s["table"], s["positions"], s["slots"], s["k_cache"], s["v_cache"],
                    q_norm=s["q_norm"], k_norm=s["k_norm"], eps=1e-6, interleaved=s["case"]["interleaved"],
                    q_out=s["q_out"], workspace=s["ws"])
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _results(s):
    return {"out": s["out"]} if s["lse"] is None else {"out": s["out"], "lse": s["lse"]}


def _own_prefill(s):
    import expert_layer_gb300 as moe
    c = s["case"]
    if c["page"]:
        moe.attn_prefill_paged(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["q_starts"], s["kv_lens"],
                               causal=c["causal"], scale=s["scale"], out=s["out"], lse=s["lse"], workspace=s["ws"])
    else:
        moe.attn_prefill(s["q"], s["k"], s["v"], s["q_starts"], s["kv_starts"], causal=c["causal"], scale=s["scale"],
                         out=s["out"], lse=s["lse"], workspace=s["ws"])
    return _results(s)


def _own_decode(s):
    import expert_layer_gb300 as moe
    moe.attn_decode(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["kv_lens"],
                    prefix_table=s.get("prefix_table"), prefix_len=s["case"]["prefix"], scale=s["scale"],
                    out=s["out"], lse=s["lse"], workspace=s["ws"])
    return _results(s)


# ------------------------------------------------------------------ the plain forms
def _rms(x, weight, eps=1e-6):
    return x if weight is None else x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * weight


def _rotate(x, cos, sin, rot, interleaved):
    head, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        a, b = head[..., 0::2], head[..., 1::2]
        head = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = head[..., :rot // 2], head[..., rot // 2:]
        head = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([head, rest], dim=-1)


def _plain_append(s):
    c = s["case"]
    angles = s["table"][s["positions"].long()][:, None, :]
    cos, sin = angles[..., :c["rot"] // 2], angles[..., c["rot"] // 2:]
    q = _rotate(_rms(s["q"].float(), s["q_norm"]), cos, sin, c["rot"], c["interleaved"])
    k = _rotate(_rms(s["k"].float(), s["k_norm"]), cos, sin, c["rot"], c["interleaved"])
    slots = s["slots"].long()
    page, row = slots // c["page"], slots % c["page"]
    s["k_cache"][page, :, row] = k.to(s["k_cache"].dtype)
    s["v_cache"][page, :, row] = s["v"]
    return {"q": q.to(s["q"].dtype), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _softmax_parts(scores):
    """(weights, log of their unnormalised sum) of masked scores; a row of -inf gets weights of 0."""
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    e = torch.exp(scores - top)
    total = e.sum(-1, keepdim=True)
    return e / torch.where(total == 0, torch.ones_like(total), total), (top + torch.log(total)).squeeze(-1)


def _unpage(cache, table, keys):
    """[n, Hkv, keys, D] of a paged cache, in 32 bits."""
    got = cache[table.long()]
    n, _, Hkv, _, D = got.shape
    return got.transpose(1, 2).reshape(n, Hkv, -1, D)[:, :, :keys].float()


def _unpack(x, starts, wide):
    """[n, heads, wide, D] of packed rows [rows, heads, D], in 32 bits; rows past a sequence's end hold others'."""
    at = starts[:-1, None].long() + torch.arange(wide, device=x.device)[None, :]
    return x[at.clamp(max=x.shape[0] - 1)].transpose(1, 2).float()


def _plain_prefill(s):
    c = s["case"]
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    group, wide, keys = Hq // Hkv, s["max_q"], s["max_kv"]
    q = _unpack(s["q"], s["q_starts"], wide)
    if c["page"]:
        k, v = _unpage(s["k_cache"], s["page_table"], keys), _unpage(s["v_cache"], s["page_table"], keys)
        kv_lens = s["kv_lens"]
    else:
        k, v = _unpack(s["k"], s["kv_starts"], keys), _unpack(s["v"], s["kv_starts"], keys)
        kv_lens = s["kv_starts"][1:] - s["kv_starts"][:-1]
    n = q.shape[0]
    q_lens = s["q_starts"][1:] - s["q_starts"][:-1]
    row, key = torch.arange(wide, device="cuda"), torch.arange(keys, device="cuda")
    seen = (key[None, None, :] < kv_lens[:, None, None]).expand(n, wide, keys)
    if c["causal"]:
        seen = seen & (key[None, None, :] <= row[None, :, None] + (kv_lens - q_lens)[:, None, None])
    scores = torch.matmul(q.reshape(n, Hkv, group * wide, D), k.transpose(-1, -2)) * s["scale"]
    scores = scores.view(n, Hkv, group, wide, keys).masked_fill_(~seen[:, None, None], -math.inf)
    weights, lse = _softmax_parts(scores)
    del scores
    out = torch.matmul(weights.view(n, Hkv, group * wide, keys), v).view(n, Hq, wide, D)
    # back to packed rows: row t of the batch belongs to the sequence whose start is the last one at or before it
    t = torch.arange(s["q"].shape[0], device="cuda")
    seq = torch.searchsorted(s["q_starts"][1:].contiguous(), t.to(torch.int32), right=True)
    at = t - s["q_starts"][seq]
    res = {"out": out[seq, :, at].to(s["q"].dtype)}
    if c["lse"]:
        res["lse"] = lse.view(n, Hq, wide)[seq, :, at]
    return res


def _plain_decode(s):
    c = s["case"]
    B, Hq, Hkv, D = c["B"], c["Hq"], c["Hkv"], c["D"]
    group = Hq // Hkv
    q = s["q"].float().view(B, Hkv, group, D)
    k, v = _unpage(s["k_cache"], s["page_table"], s["max_kv"]), _unpage(s["v_cache"], s["page_table"], s["max_kv"])
    key = torch.arange(s["max_kv"], device="cuda")
    scores = torch.matmul(q, k.transpose(-1, -2)) * s["scale"]
    scores = scores.masked_fill_((key[None, :] >= s["kv_lens"][:, None])[:, None, None], -math.inf)
    if c["prefix"]:
        # the prefix's keys meet the rows of the whole batch in one product
        pk = _unpage(s["k_cache"], s["prefix_table"][None], c["prefix"])[0]
        pv = _unpage(s["v_cache"], s["prefix_table"][None], c["prefix"])[0]
        rows = q.transpose(0, 1).reshape(Hkv, B * group, D)
        first = torch.matmul(rows, pk.transpose(-1, -2)).view(Hkv, B, group, -1).transpose(0, 1) * s["scale"]
        weights, lse = _softmax_parts(torch.cat([first, scores], dim=-1))
        head, tail = weights[..., :c["prefix"]], weights[..., c["prefix"]:]
        out = torch.matmul(tail, v)
        shared = torch.matmul(head.transpose(0, 1).reshape(Hkv, B * group, -1), pv)
        out = out + shared.view(Hkv, B, group, D).transpose(0, 1)
    else:
        weights, lse = _softmax_parts(scores)
        out = torch.matmul(weights, v)
    res = {"out": out.reshape(B, Hq, D).to(s["q"].dtype)}
    if c["lse"]:
        res["lse"] = lse.reshape(B, Hq)
    return res


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(s)
    c, scale = s["case"], 1.0 / math.sqrt(case["D"])
    lens = _lengths(case)
    q64 = s["q"].double()
    outs, lses = [], []
    at_q = at_k = 0
    group = c["Hq"] // c["Hkv"]
    for i, (nq, nk) in enumerate(lens):
        if c["page"]:
            ids = s["page_table"][i, :(nk + c["page"] - 1) // c["page"]].long()
            k = s["k_cache"][ids].double().permute(1, 0, 2, 3).flatten(1, 2)[:, :nk]
            v = s["v_cache"][ids].double().permute(1, 0, 2, 3).flatten(1, 2)[:, :nk]
            if c.get("prefix"):
                ids = s["prefix_table"].long()
                k = torch.cat([s["k_cache"][ids].double().permute(1, 0, 2, 3).flatten(1, 2)[:, :c["prefix"]], k], 1)
                v = torch.cat([s["v_cache"][ids].double().permute(1, 0, 2, 3).flatten(1, 2)[:, :c["prefix"]], v], 1)
        else:
            k = s["k"][at_k:at_k + nk].double().transpose(0, 1)
            v = s["v"][at_k:at_k + nk].double().transpose(0, 1)
        q = q64[at_q:at_q + nq]
        out = torch.empty(nq, c["Hq"], c["D"], dtype=torch.float64, device="cuda")
        lse = torch.empty(nq, c["Hq"], dtype=torch.float64, device="cuda")
        hidden = None
        if c["op"] == "prefill" and c["causal"]:
            hidden = torch.ones(nq, k.shape[1], dtype=torch.bool, device="cuda").triu(1 + k.shape[1] - nq)
        for h in range(c["Hq"]):
            logits = scale * (q[:, h] @ k[h // group].T)
            if hidden is not None:
                logits = logits.masked_fill(hidden, -math.inf)
            lse[:, h] = torch.logsumexp(logits, dim=1)
            out[:, h] = torch.softmax(logits, dim=1) @ v[h // group]
        outs.append(out)
        lses.append(lse)
        at_q += nq
        at_k += nk
    res = {"out": torch.cat(outs)}
    if c["lse"]:
        res["lse"] = torch.cat(lses)
    return res


def _exact_append(s):
    c = s["case"]
    half = c["rot"] // 2
    # the rotation as a product of complex numbers
    z = torch.complex(s["table"][:, :half].double(), s["table"][:, half:].double())[s["positions"].long()][:, None]

    def turned(x, weight):
        x = x.double()
        if weight is not None:
            x = x / torch.sqrt(x.pow(2).mean(-1, keepdim=True) + 1e-6) * weight.double()
        y = x.clone()
        if c["interleaved"]:
            w = torch.view_as_complex(x[..., :c["rot"]].reshape(*x.shape[:-1], half, 2).contiguous()) * z
            y[..., :c["rot"]] = torch.view_as_real(w).flatten(-2)
        else:
            w = torch.complex(x[..., :half], x[..., half:c["rot"]]) * z
            y[..., :half], y[..., half:c["rot"]] = w.real, w.imag
        return y

    k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
    k, v = turned(s["k"], s["k_norm"]), s["v"].double()
    slots = s["slots"].long()
    for h in range(c["Hkv"]):
        k_cache[slots // c["page"], h, slots % c["page"]] = k[:, h]
        v_cache[slots // c["page"], h, slots % c["page"]] = v[:, h]
    return {"q": turned(s["q"], s["q_norm"]), "k_cache": k_cache, "v_cache": v_cache}


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    if case["op"] == "append":
        T = case["T"]
        row = (Hq + 2 * Hkv) * D * 2
        return {"bytes": T * (2 * row + 4 * case["rot"] + 8) + (8 * D if case["norm"] else 0),
                "flops": T * (Hq + Hkv) * (3 * case["rot"] + (4 * D if case["norm"] else 0))}
    lens = _lengths(case)
    prefix = case.get("prefix", 0)
    rows, keys = sum(a for a, _ in lens), sum(b for _, b in lens) + prefix
    causal = case["op"] == "prefill" and case["causal"]
    pairs = sum(a * b - (a * (a - 1) // 2 if causal else 0) for a, b in lens) + rows * prefix
    index = 4 * (2 * len(lens) + (keys // case["page"] if case["page"] else 0))
    return {"bytes": 2 * (2 * rows * Hq * D + 2 * keys * Hkv * D) + index + (4 * rows * Hq if case["lse"] else 0),
            "flops": 4 * pairs * Hq * D}
