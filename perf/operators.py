"""The operators of the hybrid backbone's attention layers, as they are measured.

Three operators that a serving step of such a layer runs one after another:

* ``rope``    norms of queries and keys for each head with the position rotation in the same
              pass; keys and values go to the pages of the layer's cache;
* ``prompt``  causal attention over whole prompts, grouped heads, packed sequences of different
              lengths;
* ``step``    attention of one new token per sequence over the paged cache, with an optional long
              prefix that the whole batch shares.

``own = False`` computes them in elementary torch operations in 32 bits (rotation angles in 64),
rounded once at the end; ``own = True`` calls this repository's kernels.
"""
import math
import random

import torch

own = False

EPS, BASE = 1e-6, 10000.0
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}

# Bounds of the drawn cases: the largest listed case of each operator.
MOST_ROPE = 10240 * (2 * 16 + 4 * 4) * 128 * 2  # bytes
MOST_PROMPT = 10240 * 10240 * 16 * 128          # score products of the padded batch
MOST_STEP = 64 * 10240 * 4 * 128                # cache elements of the padded batch, keys alone


def listed():
    return [
        # One decode step of the benchmark's batch of 64: a launch-bound call between two layers' products.
        dict(name="rope_step", op="rope", T=64, Hq=16, Hkv=4, d=128, rot=128, dtype="bf16", page=16, far=10240, prompt=False),
        # The benchmark's long prompt, a quarter of each head rotated.
        dict(name="rope_prompt", op="rope", T=10240, Hq=16, Hkv=4, d=128, rot=32, dtype="bf16", page=64, far=10240, prompt=True),
        # fp32 heads of 64 at far positions, an odd token count, as many key heads as query heads.
        dict(name="rope_f32_far", op="rope", T=2049, Hq=16, Hkv=16, d=64, rot=64, dtype="f32", page=32, far=1000000, prompt=True),
        # A handful of short requests arriving together: the smallest prompts, down to one token.
        dict(name="prompt_short", op="prompt", N=6, lo=1, hi=200, mix=1, Hq=16, Hkv=4, d=128),
        # The benchmark's packed batch: 8 prompts of 512 to 4096 tokens.
        dict(name="prompt_varlen", op="prompt", N=8, lo=512, hi=4096, mix=2, Hq=16, Hkv=4, d=128),
        # The benchmark's long prompt.
        dict(name="prompt_10k", op="prompt", N=1, lo=10240, hi=10240, mix=3, Hq=16, Hkv=4, d=128),
        # Heads of 64, one key head per query head, a length that fills no tile.
        dict(name="prompt_d64", op="prompt", N=2, lo=2047, hi=2047, mix=4, Hq=16, Hkv=16, d=64),
        # One user's chat at 2k: the smallest step, where latency counts.
        dict(name="step_one", op="step", B=1, lo=2048, hi=2048, mix=5, Hq=16, Hkv=4, d=128, page=16, prefix=0),
        # The benchmark's decode batch over ragged caches.
        dict(name="step_batch", op="step", B=64, lo=512, hi=10240, mix=6, Hq=16, Hkv=4, d=128, page=16, prefix=0),
        # Few sequences with long caches, eight query heads on each key head: work split along the keys.
        dict(name="step_long", op="step", B=3, lo=10240, hi=40960, mix=7, Hq=16, Hkv=2, d=128, page=64, prefix=0),
        # 64 answers to one long document (a length that ends inside a page), each some way into its own.
        dict(name="step_prefix", op="step", B=64, lo=1, hi=512, mix=8, Hq=16, Hkv=4, d=128, page=16, prefix=10230),
        # A few samples from one 2k prompt, heads of 64 without groups, some with nothing of their own yet.
        dict(name="step_prefix_d64", op="step", B=13, lo=0, hi=40, mix=9, Hq=16, Hkv=16, d=64, page=32, prefix=2047),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "prompt", "step"])
    d = rng.choice([64, 128])
    G = rng.choice([1, 2, 3, 4, 5, 8, 16])
    Hkv = rng.choice([1, 2, 4, 8, 16]) if G < 8 else rng.choice([1, 2])
    Hq = G * Hkv
    page = rng.choice([16, 32, 64, 128])
    mix = rng.randrange(1 << 20)
    if op == "rope":
        dtype = rng.choice(["bf16", "f32"])
        most = MOST_ROPE // ((2 * Hq + 4 * Hkv) * d * (2 if dtype == "bf16" else 4))
        return dict(op=op, T=_log(rng, 1, max(1, min(20480, most))), Hq=Hq, Hkv=Hkv, d=d, rot=rng.choice([d, d // 2, d // 4]),
                    dtype=dtype, page=page, far=_log(rng, 2048, 1 << 20), prompt=rng.random() < 0.5)
    if op == "prompt":
        N = _log(rng, 1, 32)
        hi = _log(rng, 1, max(1, min(10240, int(math.sqrt(MOST_PROMPT / (N * Hq * d))))))
        lo = _log(rng, 1, hi)
        return dict(op=op, N=N, lo=lo, hi=hi, mix=mix, Hq=Hq, Hkv=Hkv, d=d)
    B = _log(rng, 1, 128)
    hi = _log(rng, 1, max(1, min(40960, MOST_STEP // (B * Hkv * d))))
    lo = _log(rng, 1, hi)
    prefix = _log(rng, 1, max(1, min(16384, MOST_STEP // (8 * Hkv * d)))) if rng.random() < 0.5 else 0
    return dict(op=op, B=B, lo=lo, hi=hi, mix=mix, Hq=Hq, Hkv=Hkv, d=d, page=page, prefix=prefix)


def _lengths(case):
    """The case's sequence lengths: over their logarithm where the range spans more than a factor of ten."""
    rng = random.Random(case["mix"])
    n, lo, hi = case.get("N") or case["B"], case["lo"], case["hi"]
    if lo > 0 and hi > 10 * lo:
        return [_log(rng, lo, hi) for _ in range(n)]
    return [rng.randint(lo, hi) for _ in range(n)]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    pick = random.Random(seed)
    dev = torch.device("cuda")
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    randn = lambda *shape, dtype=torch.bfloat16: torch.randn(shape, generator=gen, device=dev).to(dtype)  # noqa: E731
    s = dict(case)
    if case["op"] == "rope":
        # the fused projection's output, its q, k and v slices, and the layer's cache
        T, dtype, page = case["T"], TYPES[case["dtype"]], case["page"]
        qkv = randn(T, Hq + 2 * Hkv, d, dtype=dtype)
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        s["wq"] = 1 + 0.1 * randn(d, dtype=torch.float32)
        s["wk"] = 1 + 0.1 * randn(d, dtype=torch.float32)
        pages = -(-T // page) + 3
        order = torch.randperm(pages, generator=gen, device=dev)
        t = torch.arange(T, device=dev)
        if case["prompt"]:  # consecutive tokens of one prompt, page after page
            first = pick.randrange(max(1, case["far"] - T + 1))
            s["positions"] = (first + t).to(torch.int32)
            s["slots"] = (order[t // page] * page + t % page).to(torch.int32)
        else:  # one token of each of T sequences, anywhere in the cache
            s["positions"] = torch.randint(0, case["far"], (T,), generator=gen, device=dev, dtype=torch.int32)
            s["slots"] = torch.randperm(pages * page, generator=gen, device=dev)[:T].to(torch.int32)
        s["k_cache"] = torch.zeros((pages, Hkv, page, d), dtype=dtype, device=dev)
        s["v_cache"] = torch.zeros((pages, Hkv, page, d), dtype=dtype, device=dev)
        return s
    lens = _lengths(case)
    if case["op"] == "prompt":
        T = sum(lens)
        s["q"], s["k"] = randn(T, Hq, d), randn(T, Hkv, d)
        s["v"] = randn(T, Hq + 2 * Hkv, d)[:, Hq + Hkv:]  # where the projection left it
        s["max_len"] = max(lens)
        s["cu"] = torch.tensor([0] + lens, device=dev).cumsum(0).to(torch.int32)
        return s
    page, prefix = case["page"], case["prefix"]
    own_pages = [-(-n // page) for n in lens]
    shared = -(-prefix // page)
    total = sum(own_pages) + shared + 5
    order = list(range(total))
    pick.shuffle(order)
    table = [order[sum(own_pages[:b]):sum(own_pages[:b + 1])] for b in range(len(lens))]
    most = max(1, max(own_pages))
    s["table"] = torch.tensor([r + [-1] * (most - len(r)) for r in table], dtype=torch.int32, device=dev)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    s["prefix_pages"] = torch.tensor(order[total - shared:], dtype=torch.int32, device=dev) if prefix else None
    s["q"] = randn(case["B"], Hq, d)
    s["k_cache"], s["v_cache"] = randn(total, Hkv, page, d), randn(total, Hkv, page, d)
    return s


def _norm_rotate(x, w, positions, rot):
    """RMS norm of each head and the rotation of its first `rot` elements, pairs (i, i + rot / 2)."""
    x = x.float()
    x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w
    freq = BASE ** (torch.arange(0, rot, 2, device=x.device, dtype=torch.float64) / -rot)
    angle = positions.double()[:, None, None] * freq
    cos, sin = angle.cos().float(), angle.sin().float()
    a, b = x[..., :rot // 2], x[..., rot // 2:rot]
    return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., rot:]], dim=-1)


def _rope(s):
    dtype = s["q"].dtype
    q = _norm_rotate(s["q"], s["wq"], s["positions"], s["rot"]).to(dtype)
    k = _norm_rotate(s["k"], s["wk"], s["positions"], s["rot"]).to(dtype)
    slots = s["slots"].long()
    s["k_cache"][slots // s["page"], :, slots % s["page"]] = k
    s["v_cache"][slots // s["page"], :, slots % s["page"]] = s["v"]
    out = dict(q=q, k_cache=s["k_cache"], v_cache=s["v_cache"])
    if s["prompt"]:
        out["k"] = k
    return out


def _weights(scores, seen):
    """exp(scores) over the keys that are seen, and its sum, both after the row's maximum is taken off."""
    scores = scores.masked_fill(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    p = torch.exp(scores - top)
    return p, p.sum(-1, keepdim=True)


def _prompt(s):
    """The prompts as one padded batch."""
    q, k, v, cu, L = s["q"], s["k"], s["v"], s["cu"].long(), s["max_len"]
    Hq, Hkv, d = s["Hq"], s["Hkv"], s["d"]
    N = cu.numel() - 1
    t = torch.arange(L, device=q.device)
    inside = t < (cu[1:] - cu[:-1])[:, None]                          # [N, L]
    row = torch.where(inside, cu[:-1, None] + t, 0)
    heads = lambda x, h: x[row].float().reshape(N, L, h, -1, d).permute(0, 2, 3, 1, 4)  # noqa: E731
    qp = heads(q, Hkv)                                                # [N, Hkv, G, L, d]
    kp, vp = heads(k, Hkv), heads(v, Hkv)                             # [N, Hkv, 1, L, d]
    qp = qp.reshape(N, Hkv, -1, d)
    scores = (qp @ kp[:, :, 0].transpose(-1, -2)).mul_(d ** -0.5).reshape(N, Hkv, Hq // Hkv, L, L)
    p, l = _weights(scores, (t[None, :] <= t[:, None]))
    del scores
    o = (p.reshape(N, Hkv, -1, L) @ vp[:, :, 0]).reshape(N, Hkv, Hq // Hkv, L, d) / l
    o = o.permute(0, 3, 1, 2, 4).reshape(N, L, Hq, d)
    return o[inside].to(q.dtype)


def _step(s):
    """The sequences' pages gathered into one padded batch; the shared prefix gathered once."""
    q, page, prefix = s["q"], s["page"], s["prefix"]
    Hq, Hkv, d = s["Hq"], s["Hkv"], s["d"]
    B = q.shape[0]
    qg = q.float().reshape(B, Hkv, Hq // Hkv, d)
    table = s["table"].long().clamp(min=0)

    def gather(cache, pages):  # [..., pages] -> [..., Hkv, pages * page, d]
        return cache[pages].movedim(-3, -4).flatten(-3, -2).float()

    k, v = gather(s["k_cache"], table), gather(s["v_cache"], table)   # [B, Hkv, L, d]
    L = k.shape[2]
    scores = (qg @ k.transpose(-1, -2)) * d ** -0.5                   # [B, Hkv, G, L]
    seen = (torch.arange(L, device=q.device) < s["lens"][:, None])[:, None, None]
    if prefix:
        pk, pv = (gather(s[c], s["prefix_pages"].long())[:, :prefix] for c in ("k_cache", "v_cache"))
        by_head = qg.transpose(0, 1).reshape(Hkv, -1, d)              # [Hkv, B G, d]
        ps = (by_head @ pk.transpose(-1, -2)).mul_(d ** -0.5).reshape(Hkv, B, -1, prefix).transpose(0, 1)
        scores = torch.cat([ps, scores], dim=-1)
        seen = torch.cat([seen.new_ones((B, 1, 1, prefix)), seen], dim=-1)
    p, l = _weights(scores, seen)
    o = p[..., prefix:] @ v
    if prefix:
        po = p[..., :prefix].transpose(0, 1).reshape(Hkv, -1, prefix) @ pv
        o = o + po.reshape(Hkv, B, -1, d).transpose(0, 1)
    return (o / l.clamp(min=torch.finfo(torch.float32).tiny)).reshape(B, Hq, d).to(q.dtype)


def run(s):
    if own:
        from linear_attention_recurrent_chunked_b200 import gdn
        if s["op"] == "rope":
            q, k = gdn.qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], s["positions"], v=s["v"], rot=s["rot"], base=BASE,
                                    eps=EPS, k_cache=s["k_cache"], v_cache=s["v_cache"], slots=s["slots"], want_k=s["prompt"])
            out = dict(q=q, k_cache=s["k_cache"], v_cache=s["v_cache"])
            if s["prompt"]:
                out["k"] = k
            return out
        if s["op"] == "prompt":
            return gdn.attn_prefill(s["q"], s["k"], s["v"], s["cu"], max_len=s["max_len"])
        return gdn.attn_decode(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], prefix_pages=s["prefix_pages"],
                               prefix_len=s["prefix"])
    return dict(rope=_rope, prompt=_prompt, step=_step)[s["op"]](s)


def work(case):
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    if case["op"] == "rope":
        T, size = case["T"], 2 if case["dtype"] == "bf16" else 4
        rows = 2 * Hq + 4 * Hkv + (Hkv if case["prompt"] else 0)  # q, k, v in; q, the cache's k and v, k out
        return dict(bytes=T * rows * d * size + 8 * T + 8 * d, flops=T * (Hq + Hkv) * (4 * d + 3 * case["rot"]))
    lens = _lengths(case)
    if case["op"] == "prompt":
        return dict(bytes=sum(lens) * (2 * Hq + 2 * Hkv) * d * 2 + 4 * len(lens) + 4,
                    flops=4 * d * Hq * sum(n * (n + 1) // 2 for n in lens))
    keys, page = sum(lens) + case["prefix"], case["page"]
    pages = sum(-(-n // page) for n in lens) + -(-case["prefix"] // page)
    return dict(bytes=keys * 2 * Hkv * d * 2 + case["B"] * 2 * Hq * d * 2 + 4 * case["B"] + 4 * pages,
                flops=4 * d * Hq * (sum(lens) + case["B"] * case["prefix"]))


def exact(case, seed):
    s = prepare(case, seed)
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    if case["op"] == "rope":
        # the rotation as a product with exp(i angle)
        half = case["rot"] // 2
        i = torch.arange(half, device="cuda", dtype=torch.float64)
        angle = s["positions"].double()[:, None] * torch.exp(-i / half * math.log(BASE))
        turn = torch.polar(torch.ones_like(angle), angle)[:, None]
        out = {}
        for name, w in (("q", "wq"), ("k", "wk")):
            x = s[name].double()
            x = x / ((x * x).sum(-1, keepdim=True) / d + EPS).sqrt() * s[w].double()
            z = torch.complex(x[..., :half], x[..., half:2 * half]) * turn
            out[name] = torch.cat([z.real, z.imag, x[..., 2 * half:]], -1)
        for name, x in (("k_cache", out["k"]), ("v_cache", s["v"].double())):
            flat = torch.zeros((s[name].shape[0] * case["page"], Hkv, d), dtype=torch.float64, device="cuda")
            flat[s["slots"].long()] = x
            out[name] = flat.reshape(-1, case["page"], Hkv, d).transpose(1, 2).contiguous()
        if not case["prompt"]:
            del out["k"]
        return out
    if case["op"] == "prompt":
        o = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
        ends = s["cu"].tolist()
        for a, b in zip(ends, ends[1:]):
            ahead = torch.ones((b - a, b - a), dtype=torch.bool, device="cuda").triu(1)
            for h in range(Hq):  # one query head of one prompt at a time
                x = s["q"][a:b, h].double() @ s["k"][a:b, h * Hkv // Hq].double().T / math.sqrt(d)
                x = x.masked_fill(ahead, -math.inf)
                o[a:b, h] = (x - x.logsumexp(-1, keepdim=True)).exp() @ s["v"][a:b, h * Hkv // Hq].double()
        return o
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    shared = s["prefix_pages"].tolist() if case["prefix"] else []
    for b, n in enumerate(s["lens"].tolist()):
        def keys(cache):  # [Hkv, prefix + n, d] of this sequence
            x = cache[shared].transpose(0, 1).reshape(Hkv, -1, d)[:, :case["prefix"]]
            y = cache[s["table"][b, :-(-n // case["page"])].long()].transpose(0, 1).reshape(Hkv, -1, d)[:, :n]
            return torch.cat([x, y], 1).double()
        if n + case["prefix"]:
            x = s["q"][b].double().reshape(Hkv, -1, d) @ keys(s["k_cache"]).transpose(1, 2) / math.sqrt(d)
            o[b] = ((x - x.logsumexp(-1, keepdim=True)).exp() @ keys(s["v_cache"])).reshape(Hq, d)
    return o
