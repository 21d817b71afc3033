"""Operators around the paged key-value cache, as cases to be measured: rotary positions with several axes, a cache held
in 8 bits (append, prompts, single tokens), attention weight per key, and eviction by it.

``run`` computes an operator either in its plain form (elementary torch operations in 32 bits, rounded once at the
end) or, with ``own``, through the library's entry points.

The 8-bit cache: e4m3 codes and, for every 16 tokens of a page and key-value head, one scale for the keys and one for
the values, a power of two 2^e: the smallest with which the largest value is at most 448, -24 <= e <= 7.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
F8 = torch.float8_e4m3fn
BLOCK = 16                  # tokens that share a scale


def listed():
    return [
        # image and video tokens of a prompt: positions in time, height and width, each turning pairs of its own
        dict(name="append 3 axes 4096", op="append_axes", T=4096, Hq=32, Hkv=4, D=128, rot=128, interleaved=False,
             norm=True, page=16, axes=3, spread=False, max_pos=16384, dtype="bf16"),
        # a decode batch of the same kind of model on a small-head one: the three positions of a text token are equal
        dict(name="append 3 axes 64 f16", op="append_axes", T=64, Hq=12, Hkv=3, D=64, rot=64, interleaved=True,
             norm=False, page=64, axes=3, spread=True, max_pos=4096, dtype="f16"),
        # one token for each of 256 sequences, into blocks that are partly filled
        dict(name="append8 256 tokens", op="append8", n=256, q_low=1, q_high=1, hist=400, Hq=32, Hkv=4, D=128, rot=128,
             interleaved=False, norm=True, page=16, axes=1, spread=False, max_pos=40960, dtype="bf16", shape_seed=1),
        # a whole prefill chunk: eight prompts with what came before them
        dict(name="append8 8 prompts", op="append8", n=8, q_low=700, q_high=1300, hist=100, Hq=32, Hkv=4, D=128,
             rot=128, interleaved=False, norm=True, page=16, axes=1, spread=False, max_pos=16384, dtype="bf16",
             shape_seed=2),
        # short prompts of a small-head model behind a short history
        dict(name="prefill8 20 ragged f16", op="prefill8", n=20, q_low=1, q_high=300, hist=200, Hq=12, Hkv=3, D=64,
             causal=True, page=64, lse=False, dtype="f16", shape_seed=3),
        # chunks of long prompts: new tokens read the history of their sequence
        dict(name="prefill8 4 chunks", op="prefill8", n=4, q_low=300, q_high=1024, hist=7000, Hq=32, Hkv=4, D=128,
             causal=True, page=16, lse=True, dtype="bf16", shape_seed=4),
        # a small decode batch over short contexts: latency counts
        dict(name="decode8 8 short f16", op="decode8", B=8, kv_low=100, kv_high=700, prefix=0, Hq=16, Hkv=2, D=64,
             page=16, lse=False, dtype="f16", shape_seed=5),
        # a large decode batch over long contexts: the cache's bytes count
        dict(name="decode8 128 long", op="decode8", B=128, kv_low=2000, kv_high=8192, prefix=0, Hq=32, Hkv=4, D=128,
             page=16, lse=False, dtype="bf16", shape_seed=6),
        # what the tokens of a decode step add to their keys' weights
        dict(name="weights 64 decode", op="weights", n=64, q_low=1, q_high=1, hist=8191, Hq=32, Hkv=4, D=128, page=16,
             causal=True, dtype="bf16", shape_seed=7),
        # the last 64 tokens of long prompts as the window that judges the prompts' keys
        dict(name="weights 4 windows", op="weights", n=4, q_low=64, q_high=64, hist=16000, Hq=32, Hkv=4, D=128, page=16,
             causal=True, dtype="bf16", shape_seed=8),
        # a few short sequences of a small-head model
        dict(name="evict 8 short f16", op="evict", n=8, kv_low=100, kv_high=700, budget=128, first=4, last=32, Hkv=2,
             D=64, page=16, dtype="f16", shape_seed=9),
        # a batch of long sequences, each cut to 1024 keys
        dict(name="evict 64 long", op="evict", n=64, kv_low=200, kv_high=16384, budget=1024, first=4, last=128, Hkv=4,
             D=128, page=16, dtype="bf16", shape_seed=10),
    ]


def _log(rng, low, high):
    """A whole number between low and high, spread over the logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["append_axes", "append8", "append8", "prefill8", "prefill8", "decode8", "decode8", "weights",
                     "weights", "evict", "evict"])
    D = rng.choice([64, 128])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 4, 6, 7, 8])
    if Hq > 32:
        Hq = Hkv * 4
    page = rng.choice([16, 32, 64, 128])
    shape_seed = rng.randrange(1 << 20)
    turn = dict(rot=rng.choice([16, 32, 64, D, D]), interleaved=rng.random() < 0.4, norm=rng.random() < 0.6,
                spread=rng.random() < 0.5, max_pos=rng.choice([16384, 40960]))
    heads = dict(Hq=Hq, Hkv=Hkv, D=D, page=page, dtype=dtype)
    if op == "append_axes":
        return dict(op=op, T=_log(rng, 1, 4096), axes=rng.choice([2, 3, 4]), **turn, **heads)
    if op == "append8":
        n = _log(rng, 1, 256)
        q_high = _log(rng, 1, max(1, 8192 // n))
        return dict(op=op, n=n, q_low=max(1, q_high // rng.choice([1, 2, 50])), q_high=q_high,
                    hist=rng.choice([0, 30, 500]), axes=rng.choice([1, 1, 3]), shape_seed=shape_seed, **turn, **heads)
    if op == "prefill8":
        n = _log(rng, 1, 64)
        q_high = _log(rng, 2, int(4096 / math.sqrt(n)))
        # n * q_high * (q_high + hist) stays within the four chunks of the listed case
        hist = rng.randrange(0, max(1, min(8192, 65536 // n, 4 * 1024 * 8000 // (n * q_high) - q_high)))
        return dict(op=op, n=n, q_low=max(1, q_high // rng.choice([1, 3, 50])), q_high=q_high, hist=hist,
                    causal=rng.random() < 0.8, lse=rng.random() < 0.3, shape_seed=shape_seed, **heads)
    if op == "decode8":
        B = _log(rng, 1, 256)
        # B * kv_high * Hkv * D stays within the listed case
        kv_high = _log(rng, 16, max(16, min(131072, 128 * 4000 * 512 // (B * Hkv * D))))
        return dict(op=op, B=B, kv_low=max(1, kv_high // rng.choice([1, 4, 100])), kv_high=kv_high,
                    prefix=rng.choice([0, 0, _log(rng, 100, 16384)]), lse=rng.random() < 0.3, shape_seed=shape_seed,
                    **heads)
    if op == "weights":
        n = _log(rng, 1, 64)
        q_high = rng.choice([1, _log(rng, 2, max(2, 1024 // n))])
        # n * q_high * (q_high + hist) stays within the listed windows
        hist = rng.randrange(0, max(1, min(16384, 131072 // n, 4 * 64 * 16000 // (n * q_high) - q_high)))
        return dict(op=op, n=n, q_low=max(1, q_high // rng.choice([1, 3])), q_high=q_high, hist=hist,
                    causal=rng.random() < 0.8, shape_seed=shape_seed, **heads)
    n = _log(rng, 1, 64)
    del heads["Hq"]
    kv_high = _log(rng, 16, 16384)
    budget = _log(rng, 8, max(8, min(4096, 64 * 1024 // n)))
    first = rng.choice([0, 1, 4])
    return dict(op=op, n=n, kv_low=max(1, kv_high // rng.choice([1, 4, 100])), kv_high=kv_high, budget=budget,
                first=first, last=rng.randrange(0, budget - first), shape_seed=shape_seed, **heads)


def _lengths(case):
    """Lengths of a case's sequences: (query tokens, keys with those) for each."""
    r = random.Random(case["shape_seed"])
    if case["op"] in ("decode8", "evict"):
        return [(1, _log(r, case["kv_low"], case["kv_high"])) for _ in range(case.get("B") or case["n"])]
    q = [_log(r, case["q_low"], case["q_high"]) for _ in range(case["n"])]
    # single tokens stand behind contexts of very different lengths
    if case["op"] == "weights" and case["q_high"] == 1:
        return [(a, a + _log(r, 1, max(1, case["hist"]))) for a in q]
    return [(a, a + (r.randint(case["hist"] // 4, case["hist"]) if case["hist"] else 0)) for a in q]


def _starts(lens):
    s = [0]
    for v in lens:
        s.append(s[-1] + v)
    return s


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _pages(lens, page, gen):
    """Page lists of sequences of these lengths, scattered over a pool with a few spare pages: (table, pool size)."""
    need = [(v + page - 1) // page for v in lens]
    pool = sum(need) + 3
    order = torch.randperm(pool, generator=gen, device="cuda").to(torch.int32)
    wide = max(1, max(need))
    at = torch.tensor(_starts(need)[:-1], device="cuda")[:, None] + torch.arange(wide, device="cuda")[None, :]
    used = torch.arange(wide, device="cuda")[None, :] < torch.tensor(need, device="cuda")[:, None]
    return torch.where(used, order[at.clamp(max=pool - 1)], 0).contiguous(), pool


def _pair_axes(case):
    """The axis that turns each of the rot / 2 pairs: in runs, or taking turns."""
    half, n = case["rot"] // 2, case["axes"]
    return [i % n if case["spread"] else min(n - 1, i * n // half) for i in range(half)]


def _cache8(values, page):
    """Codes and exponents of rows [pages, Hkv, page, D]."""
    blocks = values.unflatten(2, (page // BLOCK, BLOCK))
    e = _exponent(blocks.abs().amax((3, 4)))
    return (blocks * torch.exp2(-e)[..., None, None]).clamp(-448, 448).to(F8).flatten(2, 3), e


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt, op, Hkv, D, page = DTYPES[case["dtype"]], case["op"], case["Hkv"], case["D"], case["page"]
    Hq = case.get("Hq", Hkv)

    def rand(*shape, mul=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * mul).to(dt)

    def cache8(pool):
        # keys as a head norm leaves them; values of tokens differ in size
        k = torch.randn(pool, Hkv, page, D, generator=gen, device="cuda")
        v = torch.randn(pool, Hkv, page, D, generator=gen, device="cuda")
        v = v * torch.exp2(torch.randn(pool, Hkv, page, 1, generator=gen, device="cuda"))
        (s["k_cache"], ek), (s["v_cache"], ev) = _cache8(k, page), _cache8(v, page)
        s["scales"] = torch.exp2(torch.stack([ek, ev], dim=-1)).contiguous()

    s = dict(case=case, ws=None, scale=1.0 / math.sqrt(D))
    lens = None if op == "append_axes" else _lengths(case)
    if lens is not None:
        kv = [b for _, b in lens]
        rows = sum(a for a, _ in lens)
        s["max_q"], s["max_kv"] = max(a for a, _ in lens), max(kv)
        s["q_starts"], s["kv_lens"] = _ints(_starts([a for a, _ in lens])), _ints(kv)
        s["page_table"], pool = _pages(kv, page, gen)
    else:
        rows = case["T"]
    if op in ("append_axes", "append8"):
        # q, k and v are parts of one projection's rows
        qkv = rand(rows, (Hq + 2 * Hkv) * D, mul=2.0)
        s["q"] = qkv[:, :Hq * D].view(rows, Hq, D)
        s["k"] = qkv[:, Hq * D:(Hq + Hkv) * D].view(rows, Hkv, D)
        s["v"] = qkv[:, (Hq + Hkv) * D:].view(rows, Hkv, D)
        s["q_norm"] = s["k_norm"] = None
        if case["norm"]:
            s["q_norm"] = 1.0 + 0.3 * torch.randn(D, generator=gen, device="cuda")
            s["k_norm"] = 1.0 + 0.3 * torch.randn(D, generator=gen, device="cuda")
        rot = case["rot"]
        inv = 1000000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
        angle = torch.arange(case["max_pos"], dtype=torch.float64, device="cuda")[:, None] * inv[None, :]
        s["table"] = torch.cat([angle.cos(), angle.sin()], dim=1).float().contiguous()
        s["q_out"] = torch.empty(rows, Hq, D, dtype=dt, device="cuda")
        # tokens of frames of 24 x 32 patches: time, row and column (and the frame's number once more)
        t = torch.arange(rows, device="cuda")
        first = seed % 100
        along = [t // 768 + first, t // 32 % 24 + first, t % 32 + first, t // 768]
        if case["axes"] == 1:
            s["axes"] = None
            s["positions"] = ((t + first) % case["max_pos"]).to(torch.int32)
        else:
            s["axes"] = torch.tensor(_pair_axes(case), dtype=torch.uint8, device="cuda")
            s["positions"] = torch.stack(along[:case["axes"]]).to(torch.int32)
    if op == "append_axes":
        pages = (rows + page - 1) // page + 3
        s["slots"] = torch.randperm(pages * page, generator=gen, device="cuda")[:rows].to(torch.int32)
        s["k_cache"], s["v_cache"] = rand(pages, Hkv, page, D), rand(pages, Hkv, page, D)
    elif op == "append8":
        cache8(pool)
    elif op in ("prefill8", "decode8"):
        s["q"] = rand(rows, Hq, D, mul=2.5)
        s["out"] = torch.empty(rows, Hq, D, dtype=dt, device="cuda")
        s["lse"] = torch.empty(rows, Hq, dtype=torch.float32, device="cuda") if case["lse"] else None
        if case.get("prefix"):
            n = (case["prefix"] + page - 1) // page
            s["prefix_table"] = (torch.randperm(n, generator=gen, device="cuda") + pool).to(torch.int32)
            pool += n
        cache8(pool)
    elif op == "weights":
        s["q"] = rand(rows, Hq, D, mul=2.5)
        s["k_cache"] = rand(pool, Hkv, page, D)
        scores, row, seq = _scores(s, _unpage(s["k_cache"], s["page_table"], s["max_kv"]))
        s["row_lse"] = torch.logsumexp(scores, dim=-1).flatten(1, 2)[seq, :, row].contiguous()
        del scores
        # what earlier steps left
        s["weights"] = torch.rand(case["n"], Hkv, s["max_kv"], generator=gen, device="cuda")
        s["weights"] *= torch.arange(s["max_kv"], device="cuda") < s["kv_lens"][:, None, None]
    else:
        s["out_table"] = torch.arange(case["n"] * ((case["budget"] + page - 1) // page), device="cuda")
        s["out_table"] = (s["out_table"] + pool).view(case["n"], -1).to(torch.int32)
        pool += s["out_table"].numel()
        s["k_cache"], s["v_cache"] = rand(pool, Hkv, page, D), rand(pool, Hkv, page, D)
        # accumulated attention has a heavy tail
        s["weights"] = torch.exp(2.0 * torch.randn(case["n"], Hkv, s["max_kv"], generator=gen, device="cuda"))
        s["new_weights"] = torch.empty(case["n"], Hkv, case["budget"], device="cuda")
        s["kept"] = torch.empty(case["n"], Hkv, case["budget"], dtype=torch.int32, device="cuda")
        s["new_lens"] = torch.empty(case["n"], dtype=torch.int32, device="cuda")
    if own:
        import expert_layer_gb300 as moe
        s["ws"] = moe.alloc_attn_workspace(rows, 1 if lens is None else len(lens), Hq, Hkv, D)
    return s


def run(s):
    op = s["case"]["op"]
    if own:
        return {"append_axes": _own_append, "append8": _own_append8, "prefill8": _own_prefill8,
                "decode8": _own_decode8, "weights": _own_weights, "evict": _own_evict}[op](s)
    return {"append_axes": _plain_append, "append8": _plain_append8, "prefill8": _plain_prefill8,
            "decode8": _plain_decode8, "weights": _plain_weights, "evict": _plain_evict}[op](s)


# ------------------------------------------------------------------ the library
def _own_append(s):
    import expert_layer_gb300 as moe
    moe.rope_append(s["q"], s["k"], s["v"], s["table"], s["positions"], s["slots"], s["k_cache"], s["v_cache"],
                    q_norm=s["q_norm"], k_norm=s["k_norm"], eps=1e-6, interleaved=s["case"]["interleaved"],
                    q_out=s["q_out"], workspace=s["ws"], axes=s["axes"])
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_append8(s):
    import expert_layer_gb300 as moe
    moe.rope_append_fp8(s["q"], s["k"], s["v"], s["table"], s["positions"], s["page_table"], s["q_starts"],
                        s["kv_lens"], s["k_cache"], s["v_cache"], s["scales"], q_norm=s["q_norm"], k_norm=s["k_norm"],
                        eps=1e-6, interleaved=s["case"]["interleaved"], axes=s["axes"], q_out=s["q_out"],
                        workspace=s["ws"])
    # (codes are values in units of their scale)
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"], "scales": s["scales"]}


def _results(s):
    return {"out": s["out"]} if s["lse"] is None else {"out": s["out"], "lse": s["lse"]}


def _own_prefill8(s):
    import expert_layer_gb300 as moe
    moe.attn_prefill_paged_fp8(s["q"], s["k_cache"], s["v_cache"], s["scales"], s["page_table"], s["q_starts"],
                               s["kv_lens"], causal=s["case"]["causal"], scale=s["scale"], out=s["out"], lse=s["lse"],
                               workspace=s["ws"])
    return _results(s)


def _own_decode8(s):
    import expert_layer_gb300 as moe
    moe.attn_decode_fp8(s["q"], s["k_cache"], s["v_cache"], s["scales"], s["page_table"], s["kv_lens"],
                        prefix_table=s.get("prefix_table"), prefix_len=s["case"]["prefix"], scale=s["scale"],
                        out=s["out"], lse=s["lse"], workspace=s["ws"])
    return _results(s)


def _own_weights(s):
    import expert_layer_gb300 as moe
    moe.attn_key_weights(s["q"], s["k_cache"], s["page_table"], s["q_starts"], s["kv_lens"], s["row_lse"],
                         s["weights"], causal=s["case"]["causal"], scale=s["scale"], workspace=s["ws"])
    return {"weights": s["weights"]}


def _own_evict(s):
    import expert_layer_gb300 as moe
    c = s["case"]
    moe.kv_evict(s["k_cache"], s["v_cache"], s["page_table"], s["kv_lens"], s["weights"], s["out_table"], c["budget"],
                 keep_first=c["first"], keep_last=c["last"], new_lens=s["new_lens"], new_weights=s["new_weights"],
                 kept=s["kept"], workspace=s["ws"])
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "new_lens": s["new_lens"],
            "new_weights": s["new_weights"], "kept": s["kept"]}


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


def _turned(s):
    """Normed and rotated queries and keys, in 32 bits."""
    c = s["case"]
    half = c["rot"] // 2
    pos = s["positions"].long()
    if s["axes"] is None:
        cos, sin = s["table"][pos, :half], s["table"][pos, half:]
    else:
        at = pos[s["axes"].long()].T                       # [T, pairs]: the position that turns each pair
        pair = torch.arange(half, device="cuda")[None, :]
        cos, sin = s["table"][at, pair], s["table"][at, pair + half]
    cos, sin = cos[:, None, :], sin[:, None, :]
    return (_rotate(_rms(s["q"].float(), s["q_norm"]), cos, sin, c["rot"], c["interleaved"]),
            _rotate(_rms(s["k"].float(), s["k_norm"]), cos, sin, c["rot"], c["interleaved"]))


def _plain_append(s):
    c = s["case"]
    q, k = _turned(s)
    slots = s["slots"].long()
    page, row = slots // c["page"], slots % c["page"]
    s["k_cache"][page, :, row] = k.to(s["k_cache"].dtype)
    s["v_cache"][page, :, row] = s["v"]
    return {"q": q.to(s["q"].dtype), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _exponent(top):
    """The smallest e with top <= 448 * 2^e, -24 <= e <= 7."""
    m, e = torch.frexp(top)                                # top = m * 2^e, 0.5 <= m < 1, and 448 = 0.875 * 2^9
    e = torch.where(m <= 0.875, e - 9, e - 8).float()
    return torch.where(top == 0, torch.full_like(e, -24), e).clamp(-24, 7)


def _rows_of(s):
    """Sequence and place within it of every packed row."""
    t = torch.arange(s["q"].shape[0], device="cuda")
    seq = torch.searchsorted(s["q_starts"][1:].contiguous(), t.to(torch.int32), right=True)
    return seq, t - s["q_starts"][seq]


def _plain_append8(s):
    c = s["case"]
    page, Hkv, D = c["page"], c["Hkv"], c["D"]
    q, k = _turned(s)
    seq, i = _rows_of(s)
    before = s["kv_lens"] - (s["q_starts"][1:] - s["q_starts"][:-1])       # tokens that were there
    at = (before[seq] + i).long()
    where = s["page_table"][seq, at // page].long()
    block, row = where * (page // BLOCK) + at % page // BLOCK, at % BLOCK   # scale blocks of the whole cache, in a line
    blocks = s["scales"].shape[0] * (page // BLOCK)
    # blocks that hold rows of before: the first one of each sequence whose first new row is not its first
    old_rows = torch.zeros(blocks, dtype=torch.int64, device="cuda")
    old_rows[block[s["q_starts"][:-1].long()]] = before.long() % BLOCK
    touched = torch.zeros(blocks, dtype=torch.bool, device="cuda")
    touched[block] = True
    old_e = torch.log2(s["scales"]).permute(0, 2, 1, 3).reshape(blocks, Hkv, 2)
    new_e = old_e.clone()
    for x, name, values in ((0, "k_cache", k), (1, "v_cache", s["v"].float())):
        top = torch.zeros(blocks, Hkv, device="cuda")
        top.scatter_reduce_(0, block[:, None].expand(-1, Hkv), values.abs().amax(-1), "amax")
        need = _exponent(top)
        e = torch.where((old_rows > 0)[:, None], torch.maximum(need, old_e[..., x]), need)
        e = torch.where(touched[:, None], e, old_e[..., x])
        new_e[..., x] = e
        # [blocks, Hkv, 16, D] of the codes; rows of before in units of the new scale
        codes = s[name].view(torch.uint8).unflatten(2, (page // BLOCK, BLOCK)).transpose(1, 2).reshape(blocks, Hkv, BLOCK, D)
        first = block[s["q_starts"][:-1].long()]
        f = torch.exp2(old_e[first, :, x] - e[first])[..., None, None]
        again = (codes[first].view(F8).float() * f).to(F8).view(torch.uint8)
        kept = torch.arange(BLOCK, device="cuda")[None, :] < old_rows[first][:, None]
        codes[first] = torch.where(kept[:, None, :, None], again, codes[first])
        mine = (values * torch.exp2(-e[block])[..., None]).clamp(-448, 448).to(F8).view(torch.uint8)
        codes[block, :, row] = mine
        back = codes.view(-1, page // BLOCK, Hkv, BLOCK, D).transpose(1, 2).reshape(s[name].shape)
        s[name].copy_(back.view(F8))
    s["scales"].copy_(torch.exp2(new_e).view(-1, page // BLOCK, Hkv, 2).permute(0, 2, 1, 3))
    return {"q": q.to(s["q"].dtype), "k_cache": s["k_cache"], "v_cache": s["v_cache"], "scales": s["scales"]}


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


def _unpage8(s, name, table, keys):
    """The same of a cache in 8 bits."""
    got = s[name].view(torch.uint8)[table.long()].view(F8).float()        # [n, pages, Hkv, page, D]
    scale = s["scales"][..., 0 if name == "k_cache" else 1][table.long()]
    got = got * scale.repeat_interleave(BLOCK, dim=3)[..., None]
    n, _, Hkv, _, D = got.shape
    return got.transpose(1, 2).reshape(n, Hkv, -1, D)[:, :, :keys]


def _scores(s, k):
    """Masked logits [n, Hkv, group, wide, keys], and the place and sequence of every packed row."""
    c = s["case"]
    n, Hkv, keys, D = k.shape
    wide, group = s["max_q"], c["Hq"] // Hkv
    at = s["q_starts"][:-1, None].long() + torch.arange(wide, device="cuda")[None, :]
    q = s["q"][at.clamp(max=s["q"].shape[0] - 1)].transpose(1, 2).float()      # [n, Hq, wide, D]
    q_lens = s["q_starts"][1:] - s["q_starts"][:-1]
    row, key = torch.arange(wide, device="cuda"), torch.arange(keys, device="cuda")
    seen = (key[None, None, :] < s["kv_lens"][:, None, None]).expand(n, wide, keys)
    if c["causal"]:
        seen = seen & (key[None, None, :] <= row[None, :, None] + (s["kv_lens"] - q_lens)[:, None, None])
    scores = torch.matmul(q.reshape(n, Hkv, group * wide, D), k.transpose(-1, -2)) * s["scale"]
    scores = scores.view(n, Hkv, group, wide, keys).masked_fill_(~seen[:, None, None], -math.inf)
    seq, place = _rows_of(s)
    return scores, place, seq


def _plain_prefill8(s):
    c = s["case"]
    k, v = (_unpage8(s, name, s["page_table"], s["max_kv"]) for name in ("k_cache", "v_cache"))
    scores, place, seq = _scores(s, k)
    n, Hkv, group, wide, keys = scores.shape
    weights, lse = _softmax_parts(scores)
    del scores
    out = torch.matmul(weights.view(n, Hkv, group * wide, keys), v).view(n, c["Hq"], wide, c["D"])
    res = {"out": out[seq, :, place].to(s["q"].dtype)}
    if c["lse"]:
        res["lse"] = lse.view(n, c["Hq"], wide)[seq, :, place]
    return res


def _plain_decode8(s):
    c = s["case"]
    B, Hq, Hkv, D = c["B"], c["Hq"], c["Hkv"], c["D"]
    group = Hq // Hkv
    q = s["q"].float().view(B, Hkv, group, D)
    k, v = (_unpage8(s, name, s["page_table"], s["max_kv"]) for name in ("k_cache", "v_cache"))
    key = torch.arange(s["max_kv"], device="cuda")
    scores = torch.matmul(q, k.transpose(-1, -2)) * s["scale"]
    scores = scores.masked_fill_((key[None, :] >= s["kv_lens"][:, None])[:, None, None], -math.inf)
    if c["prefix"]:
        # the prefix's keys meet the rows of the whole batch in one product
        pk, pv = (_unpage8(s, name, s["prefix_table"][None], c["prefix"])[0] for name in ("k_cache", "v_cache"))
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


def _plain_weights(s):
    scores, place, seq = _scores(s, _unpage(s["k_cache"], s["page_table"], s["max_kv"]))
    n, Hkv, group, wide, keys = scores.shape
    # log-sums as [n, Hkv, group, wide]; places past a sequence's end count for nothing
    lse = torch.full((n, wide, Hkv * group), math.inf, device="cuda")
    lse[seq, place] = s["row_lse"]
    p = torch.exp(scores - lse.transpose(1, 2).reshape(n, Hkv, group, wide, 1))
    s["weights"] += p.sum((2, 3))
    return {"weights": s["weights"]}


def _plain_evict(s):
    c = s["case"]
    n, budget, page = c["n"], c["budget"], c["page"]
    lens = s["kv_lens"].long()
    key = torch.arange(s["max_kv"], device="cuda")
    inside = key[None, :] < lens[:, None]
    always = inside & ((key < c["first"]) | (key >= (lens - c["last"])[:, None]))
    rank = torch.where(always[:, None, :], math.inf, s["weights"])
    rank = torch.where(inside[:, None, :], rank, -math.inf)
    # a stable sort: of equal weights the first key
    order = rank.sort(dim=-1, descending=True, stable=True).indices[..., :budget]
    new_lens = lens.clamp(max=budget)
    used = torch.arange(order.shape[-1], device="cuda")[None, :] < new_lens[:, None]
    kept = torch.where(used[:, None, :], order, s["max_kv"]).sort(-1).values
    kept = torch.nn.functional.pad(kept, (0, budget - kept.shape[-1]), value=s["max_kv"])
    here = kept < s["max_kv"]
    at = kept.clamp(max=s["max_kv"] - 1)
    seq, head, j = here.nonzero(as_tuple=True)
    src, j_page = at[seq, head, j], s["out_table"][seq, j // page].long()
    for cache in (s["k_cache"], s["v_cache"]):
        cache[j_page, head, j % page] = cache[s["page_table"][seq, src // page].long(), head, src % page]
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "new_lens": new_lens.to(torch.int32),
            "new_weights": torch.where(here, s["weights"].gather(-1, at), 0.0),
            "kept": torch.where(here, kept, -1).to(torch.int32)}


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"append_axes": _exact_append, "append8": _exact_append8, "prefill8": _exact_attention,
            "decode8": _exact_attention, "weights": _exact_weights, "evict": _exact_evict}[case["op"]](s)


def _complex_turned(s, x, weight):
    """Normed rows, their pairs multiplied by complex numbers of the positions' angles."""
    c = s["case"]
    half = c["rot"] // 2
    z = torch.empty(x.shape[0], half, dtype=torch.complex128, device="cuda")
    for i in range(half):
        pos = s["positions"] if s["axes"] is None else s["positions"][int(s["axes"][i])]
        row = s["table"][pos.long()].double()
        z[:, i] = torch.complex(row[:, i], row[:, half + i])
    z = z[:, None]
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


def _exact_append(s):
    c = s["case"]
    k, v = _complex_turned(s, s["k"], s["k_norm"]), s["v"].double()
    k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
    slots = s["slots"].long()
    for h in range(c["Hkv"]):
        k_cache[slots // c["page"], h, slots % c["page"]] = k[:, h]
        v_cache[slots // c["page"], h, slots % c["page"]] = v[:, h]
    return {"q": _complex_turned(s, s["q"], s["q_norm"]), "k_cache": k_cache, "v_cache": v_cache}


def _round8(x):
    """To the nearest e4m3 value, ties to even, at most 448 (64 bits)."""
    step = torch.exp2((torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -9))) - 3).clamp(min=-9))
    return (torch.round(x / step) * step).clamp(-448, 448)


def _exact_append8(s):
    c = s["case"]
    page = c["page"]
    k, v = _complex_turned(s, s["k"], s["k_norm"]), s["v"].double()
    scales = s["scales"].double()
    caches = [s["k_cache"].double(), s["v_cache"].double()]
    ladder = torch.exp2(torch.arange(-24, 8, dtype=torch.float64, device="cuda"))
    t = 0
    for i, (n, kv) in enumerate(_lengths(c)):
        table = s["page_table"][i].tolist()
        at = kv - n
        while at < kv:
            to = min(kv, at // BLOCK * BLOCK + BLOCK)
            p, first = table[at // page], at % page // BLOCK * BLOCK
            r0, r1 = at % page, at % page + to - at
            for x, rows in enumerate((k[t:t + to - at], v[t:t + to - at])):
                cache = caches[x][p]
                top = rows.abs().amax((0, 2))
                scale = ladder[(448 * ladder[None, :] < top[:, None]).sum(1).clamp(max=31)]
                if r0 > first:
                    old = scales[p, :, first // BLOCK, x].clone()
                    scale = torch.maximum(scale, old)
                    cache[:, first:r0] = _round8(cache[:, first:r0] * (old / scale)[:, None, None])
                scales[p, :, first // BLOCK, x] = scale
                cache[:, r0:r1] = _round8(rows.transpose(0, 1) / scale[:, None, None])
            t += to - at
            at = to
    return {"q": _complex_turned(s, s["q"], s["q_norm"]), "k_cache": caches[0], "v_cache": caches[1], "scales": scales}


def _exact_rows(s, name, table, n):
    """The first n rows [Hkv, n, D] of a page list."""
    ids = table[:(n + s["case"]["page"] - 1) // s["case"]["page"]].long()
    if s["k_cache"].dtype == F8:
        rows = s[name].view(torch.uint8)[ids].view(F8).double()
        scale = s["scales"][ids][..., 0 if name == "k_cache" else 1].double()
        rows = (rows.unflatten(2, (-1, BLOCK)) * scale[..., None, None]).flatten(2, 3)
    else:
        rows = s[name][ids].double()
    return rows.permute(1, 0, 2, 3).flatten(1, 2)[:, :n]


def _exact_attention(s):
    c = s["case"]
    outs, lses = [], []
    at, group = 0, c["Hq"] // c["Hkv"]
    q64 = s["q"].double()
    for i, (nq, nk) in enumerate(_lengths(c)):
        k, v = (_exact_rows(s, name, s["page_table"][i], nk) for name in ("k_cache", "v_cache"))
        if c.get("prefix"):
            k = torch.cat([_exact_rows(s, "k_cache", s["prefix_table"], c["prefix"]), k], 1)
            v = torch.cat([_exact_rows(s, "v_cache", s["prefix_table"], c["prefix"]), v], 1)
        hidden = None
        if c["op"] == "prefill8" and c["causal"]:
            hidden = torch.ones(nq, k.shape[1], dtype=torch.bool, device="cuda").triu(1 + k.shape[1] - nq)
        out = torch.empty(nq, c["Hq"], c["D"], dtype=torch.float64, device="cuda")
        lse = torch.empty(nq, c["Hq"], dtype=torch.float64, device="cuda")
        for h in range(c["Hq"]):
            logits = q64[at:at + nq, h] @ k[h // group].T / math.sqrt(c["D"])
            if hidden is not None:
                logits = logits.masked_fill(hidden, -math.inf)
            lse[:, h] = torch.logsumexp(logits, dim=1)
            out[:, h] = torch.softmax(logits, dim=1) @ v[h // group]
        outs.append(out)
        lses.append(lse)
        at += nq
    res = {"out": torch.cat(outs)}
    if c["lse"]:
        res["lse"] = torch.cat(lses)
    return res


def _exact_weights(s):
    c = s["case"]
    weights = s["weights"].double()
    at, group = 0, c["Hq"] // c["Hkv"]
    for i, (nq, nk) in enumerate(_lengths(c)):
        k = _exact_rows(s, "k_cache", s["page_table"][i], nk)
        for h in range(c["Hq"]):
            logits = s["q"][at:at + nq, h].double() @ k[h // group].T / math.sqrt(c["D"])
            p = torch.exp(logits - s["row_lse"][at:at + nq, h].double()[:, None])
            weights[i, h // group, :nk] += (p.tril(nk - nq) if c["causal"] else p).sum(0)
        at += nq
    return {"weights": weights}


def _exact_evict(s):
    c = s["case"]
    page, budget = c["page"], c["budget"]
    k_cache, v_cache = s["k_cache"].clone(), s["v_cache"].clone()
    kept = torch.full((c["n"], c["Hkv"], budget), -1, dtype=torch.int32)
    new_weights = torch.zeros(c["n"], c["Hkv"], budget, dtype=torch.float64)
    new_lens = []
    weights, lens = s["weights"].cpu(), [b for _, b in _lengths(c)]
    for i, n in enumerate(lens):
        new_lens.append(min(n, budget))
        for h in range(c["Hkv"]):
            keep = list(range(n))
            if n > budget:
                middle = range(c["first"], n - c["last"])
                w = weights[i, h].tolist()
                best = sorted(middle, key=lambda j: (-w[j], j))[:budget - c["first"] - c["last"]]
                keep = list(range(c["first"])) + sorted(best) + list(range(n - c["last"], n))
            kept[i, h, :len(keep)] = torch.tensor(keep, dtype=torch.int32)
            src = torch.tensor(keep, device="cuda")
            j = torch.arange(len(keep), device="cuda")
            frm, to = s["page_table"][i, src // page].long(), s["out_table"][i, j // page].long()
            for new, old in ((k_cache, s["k_cache"]), (v_cache, s["v_cache"])):
                new[to, h, j % page] = old[frm, h, src % page]
            new_weights[i, h, :len(keep)] = weights[i, h, keep].double()
    return {"k_cache": k_cache.double(), "v_cache": v_cache.double(), "new_lens": _ints(new_lens),
            "new_weights": new_weights.cuda(), "kept": kept.cuda()}


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    Hkv, D = case["Hkv"], case["D"]
    Hq = case.get("Hq", 0)
    op = case["op"]
    if op in ("append_axes", "append8"):
        T = case["T"] if op == "append_axes" else sum(a for a, _ in _lengths(case))
        stored = 2 * Hkv * D * (2 if op == "append_axes" else 1)
        read = (Hq + 2 * Hkv) * D * 2 + 4 * case["rot"] + 4 * case["axes"] + 4
        return {"bytes": T * (read + Hq * D * 2 + stored) + (8 * D if case["norm"] else 0),
                "flops": T * (Hq + Hkv) * (3 * case["rot"] + (4 * D if case["norm"] else 0))}
    lens = _lengths(case)
    rows, keys = sum(a for a, _ in lens), sum(b for _, b in lens)
    causal = op in ("prefill8", "weights") and case["causal"]
    pairs = sum(a * b - (a * (a - 1) // 2 if causal else 0) for a, b in lens)
    index = 4 * (2 * len(lens) + keys // case["page"])
    if op == "evict":
        moved = sum(min(b, case["budget"]) for _, b in lens)
        return {"bytes": 4 * keys * Hkv + moved * Hkv * (2 * 2 * D * 2 + 8) + index, "flops": 0}
    if op == "weights":
        return {"bytes": 2 * rows * Hq * D + 4 * rows * Hq + 2 * keys * Hkv * D + 8 * keys * Hkv + index,
                "flops": 2 * pairs * Hq * D}
    prefix = case.get("prefix", 0)
    keys, pairs = keys + prefix, pairs + rows * prefix
    return {"bytes": 2 * 2 * rows * Hq * D + 2 * keys * Hkv * D + 8 * (keys // BLOCK) * Hkv + index
            + (4 * rows * Hq if case["lse"] else 0),
            "flops": 4 * pairs * Hq * D}
