"""The serving operators around a prompt and its 8-bit cache, as a user's program calls them.

Five operators that a server runs one after the other for each layer: attention over packed prompts (output and
row log-sum-exp only), the attention weight that every key of those prompts received, writing keys and values into a
paged 8-bit cache, attention over that cache, and the eviction of the cached tokens that received least weight.

With ``own`` false, ``run`` computes them from elementary torch operations in float32, rounded once at the end; with
``own`` true it makes the calls of ``sdpa_forward_materialised_amd``. ``exact`` computes them again in float64, one
sequence and head at a time.

Cache: pages of ``page`` tokens. k codes [pages, Hkv, page, D] and v codes [pages, Hkv, D, page] in e4m3, one float32
scale (a power of two) per page and head for each of k and v. A page table row lists a sequence's pages in order.
"""

import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
E4M3 = torch.float8_e4m3fn
TOP = 448.0  # the largest e4m3 value


# ---------------------------------------------------------------------------------------------------------- the cases

def listed():
    return [
        # the smallest prompt a server sees: one short question, two heads, float32 (the framework's check shape)
        dict(name="prompt_64_f32", op="prompt", lens="64", Hq=2, Hkv=2, D=32, dtype="f32"),
        # a batch of ragged prompts, a one-token one among them, grouped heads, head dim 64, fp16
        dict(name="prompt_ragged_1k_f16", op="prompt", lens="1024,700,1,333,1000", Hq=8, Hkv=2, D=64, dtype="f16"),
        # long documents of odd lengths, grouped heads of 128, bf16: the largest prompt work
        dict(name="prompt_12k_bf16", op="prompt", lens="12289,5003", Hq=16, Hkv=4, D=128, dtype="bf16"),
        # weights that an eviction of a 2k-token prompt goes by: every head has its own keys, bf16
        dict(name="weights_2k_bf16", op="weights", lens="2048,1531", Hq=16, Hkv=16, D=128, dtype="bf16"),
        # the same for a long fp16 document with four query heads to a key head
        dict(name="weights_8k_f16", op="weights", lens="8191", Hq=16, Hkv=4, D=64, dtype="f16"),
        # one new token for each of 16 sequences in their decode loop, pages of 64
        dict(name="append_16x1_bf16", op="append", before="4095,17,64,1000", repeat=4, new="1", Hkv=8, D=128, page=64,
             dtype="bf16"),
        # whole prompts written after an attention over them, ragged, pages of 16
        dict(name="append_prompts_f16", op="append", before="0,0,40,7", repeat=2, new="4096,3001,512,2047", Hkv=8, D=128,
             page=16, dtype="f16"),
        # one short conversation's next token: latency counts
        dict(name="cache_1x200_f16", op="cache", lens="200", repeat=1, new=1, Hq=8, Hkv=2, D=64, page=16, weigh=False,
             dtype="f16"),
        # a full batch's next tokens, ragged caches, four query heads to a key head, weights gathered for an eviction
        dict(name="cache_16x4k_weigh_bf16", op="cache", lens="4096,3500,1111,2900", repeat=4, new=1, Hq=32, Hkv=8, D=128,
             page=64, weigh=True, dtype="bf16"),
        # long contexts' chunks of 8 tokens (drafted tokens to be checked at once): the largest cache
        dict(name="cache_4x32k_chunk_bf16", op="cache", lens="32768,30001", repeat=2, new=8, Hq=32, Hkv=8, D=128, page=64,
             weigh=False, dtype="bf16"),
        # a batch of filled caches cut to a quarter
        dict(name="evict_16x4k", op="evict", lens="4096,3500,1111,2900", repeat=4, Hkv=8, D=128, page=64, budget=1024,
             recent=128),
        # one long cache cut to an eighth, small pages
        dict(name="evict_1x32k", op="evict", lens="32768", repeat=1, Hkv=8, D=128, page=16, budget=4096, recent=512),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng: random.Random):
    op = rng.choice(["prompt", "weights", "append", "cache", "evict"])
    D = rng.choice([32, 64, 128])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 2, 3, 4, 7, 8])
    page = rng.choice([16, 32, 64, 128])
    if op in ("prompt", "weights"):
        top = _spread(rng, 64, 6000)
        lens = [top] + [rng.randint(0, top) for _ in range(rng.choice([0, 1, 3, 5]))]
        Hq = Hkv * group
        while Hq > Hkv and len(lens) * top * top * Hq > 3.0e9:  # the padded scores of the plain form
            group = max(1, group // 2)
            Hq = Hkv * group
        while len(lens) * top * top * Hq > 3.0e9:
            lens = lens[:-1] if len(lens) > 1 else [top // 2 + 1]
            top = max(lens)
        return dict(op=op, lens=",".join(map(str, lens)), Hq=Hq, Hkv=Hkv, D=D,
                    dtype=rng.choice(["f16", "bf16"] if top > 1500 else ["f32", "f16", "bf16"]))
    if op == "append":
        n = rng.randint(1, 4)
        most = 1 if rng.random() < 0.4 else _spread(rng, 2, 4000)
        return dict(op=op, before=",".join(str(rng.randint(0, 4000)) for _ in range(n)), repeat=rng.choice([1, 2, 4]),
                    new=",".join(str(rng.randint(1, most)) for _ in range(n)), Hkv=Hkv, D=D, page=page,
                    dtype=rng.choice(["f16", "bf16"]))
    top = _spread(rng, 100, 32000)
    lens = [top] + [rng.randint(1, top) for _ in range(rng.choice([0, 1, 3]))]
    repeat = rng.choice([1, 2, 4])
    while repeat > 1 and repeat * len(lens) * top * Hkv * D > 125e6:
        repeat //= 2
    while len(lens) > 1 and len(lens) * top * Hkv * D > 125e6:
        lens = lens[:-1]
    lens = ",".join(map(str, lens))
    if op == "cache":
        return dict(op=op, lens=lens, repeat=repeat, new=rng.choice([1, 1, 1, 2, 5, 8]), Hq=Hkv * group, Hkv=Hkv, D=D,
                    page=page, weigh=rng.random() < 0.5, dtype=rng.choice(["f16", "bf16"]))
    budget = rng.randint(max(1, top // 16), max(1, top - top // 8))
    return dict(op=op, lens=lens, repeat=repeat, Hkv=Hkv, D=D, page=page, budget=budget,
                recent=rng.randint(0, max(0, budget // 2)))


def _ints(text):
    return [int(x) for x in text.split(",")]


def work(case):
    c = case
    if c["op"] in ("prompt", "weights"):
        lens, es = _ints(c["lens"]), 4 if c["dtype"] == "f32" else 2
        T, pairs = sum(lens), sum(n * (n + 1) // 2 for n in lens)
        if c["op"] == "prompt":
            return {"bytes": T * c["D"] * es * 2 * (c["Hq"] + c["Hkv"]) + 4 * T * c["Hq"], "flops": 4 * c["D"] * c["Hq"] * pairs}
        return {"bytes": T * c["D"] * es * (c["Hq"] + c["Hkv"]) + 4 * T * c["Hq"] + 4 * len(lens) * c["Hkv"] * max(lens),
                "flops": 2 * c["D"] * c["Hq"] * pairs}
    if c["op"] == "append":
        new, before = _ints(c["new"]), _ints(c["before"])
        T = sum(new[i % len(new)] for i in range(len(before))) * c["repeat"]
        return {"bytes": 2 * T * c["Hkv"] * c["D"] * 3, "flops": 0}
    lens = _ints(c["lens"]) * c["repeat"]
    if c["op"] == "cache":
        live = sum(lens)
        rows = c["new"] * len(lens)
        pairs = sum(max(0, n - i) for n in lens for i in range(c["new"]))
        return {"bytes": 2 * live * c["Hkv"] * c["D"] + 2 * 2 * rows * c["Hq"] * c["D"] + 4 * rows * c["Hq"] +
                (8 * live * c["Hkv"] if c["weigh"] else 0), "flops": 4 * c["D"] * c["Hq"] * pairs}
    kept = sum(min(n, c["budget"]) for n in lens)
    return {"bytes": c["Hkv"] * (4 * sum(lens) + 4 * kept * c["D"] + 4 * kept + 4 * len(lens) * c["budget"]), "flops": 0}


# --------------------------------------------------------------------------------------------------------- the inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _qkv(g, T, Hq, Hkv, D, dtype):
    """Queries and keys of which some scores stand out (a channel pattern that the keys share), plain values."""
    lean = _normal(g, 1, Hkv, D)
    q = (1.5 * _normal(g, T, Hq, D)).to(dtype)
    k = (_normal(g, T, Hkv, D) + lean).to(dtype)
    v = _normal(g, T, Hkv, D).to(dtype)
    return q, k, v


def _cu(lens):
    return torch.tensor([0] + lens, device=DEV).cumsum(0).to(torch.int32)


def _pages(g, counts, spare=2):
    """Page table rows for sequences of `counts` pages, in shuffled order, and the number of pages of the pool."""
    n = sum(counts) + spare
    order = torch.randperm(n, generator=g, device=DEV).to(torch.int32)
    wide = max(1, max(counts))
    first = torch.tensor([0] + counts[:-1], device=DEV).cumsum(0)
    at = first[:, None] + torch.arange(wide, device=DEV)[None, :]
    full = torch.arange(wide, device=DEV)[None, :] < torch.tensor(counts, device=DEV)[:, None]
    return torch.where(full, order[at.clamp(max=n - 1)], torch.zeros_like(order[:1])), n


def _filled(g, n_pages, Hkv, page, D):
    """A pool whose pages hold codes of the whole e4m3 range under scales as normal keys and values get them."""
    k = (_normal(g, n_pages, Hkv, page, D) * 130).clamp(-TOP, TOP).to(E4M3)
    v = (_normal(g, n_pages, Hkv, D, page) * 130).clamp(-TOP, TOP).to(E4M3)
    ks, vs = (torch.exp2(torch.randint(-8, -5, (n_pages, Hkv), generator=g, device=DEV).float()) for _ in range(2))
    return [k, v, ks, vs]


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = dict(case)
    if c["op"] in ("prompt", "weights"):
        lens = _ints(c["lens"])
        s["cu"], s["most"] = _cu(lens), max(lens)
        s["q"], s["k"], s["v"] = _qkv(g, sum(lens), c["Hq"], c["Hkv"], c["D"], TYPES[c["dtype"]])
        if c["op"] == "weights":  # the row log-sum-exp that the attention before it returned
            s["lse"] = _lse(s)
        return s
    if c["op"] == "append":
        before, new = _ints(c["before"]), _ints(c["new"])
        new = [new[i % len(new)] for i in range(len(before))] * c["repeat"]
        before = before * c["repeat"]
        table, n = _pages(g, [-(-(b + m) // c["page"]) for b, m in zip(before, new)])
        s["cache"], s["table"] = _filled(g, n, c["Hkv"], c["page"], c["D"]), table
        s["lens"] = torch.tensor(before, device=DEV, dtype=torch.int32)
        s["cu"], s["most"] = _cu(new), max(new)
        _, s["k"], s["v"] = _qkv(g, sum(new), 1, c["Hkv"], c["D"], TYPES[c["dtype"]])
        return s
    lens = _ints(c["lens"]) * c["repeat"]
    s["lens"], s["most_kv"] = torch.tensor(lens, device=DEV, dtype=torch.int32), max(lens)
    counts = [-(-n // c["page"]) for n in lens]
    if c["op"] == "cache":
        table, n = _pages(g, counts)
        s["cache"], s["table"] = _filled(g, n, c["Hkv"], c["page"], c["D"]), table
        s["cu"] = _cu([c["new"]] * len(lens))
        s["q"] = (_normal(g, c["new"] * len(lens), c["Hq"], c["D"])).to(TYPES[c["dtype"]])
        if c["weigh"]:
            s["weights"] = _normal(g, len(lens), c["Hkv"], max(lens)).abs()
            s["weights_out"] = torch.zeros_like(s["weights"])
        return s
    to = [-(-min(n, c["budget"]) // c["page"]) for n in lens]
    table, n = _pages(g, [a + b for a, b in zip(counts, to)])
    # a sequence's present pages come first in its row, the pages it moves to behind them
    at = torch.tensor(counts, device=DEV)[:, None] + torch.arange(max(to), device=DEV)[None, :]
    s["to"] = table.gather(1, at.clamp(max=table.shape[1] - 1)).contiguous()
    s["table"] = table[:, :max(counts)].contiguous()
    s["cache"] = _filled(g, n, c["Hkv"], c["page"], c["D"])
    s["weights"] = _normal(g, len(lens), c["Hkv"], max(lens)).abs().pow(3)
    s["weights_out"] = torch.zeros_like(s["weights"])
    return s


def _pool(s):
    """The cache object over the pool's tensors, built once as a server builds it."""
    if "pool" not in s:
        import sdpa_forward_materialised_amd as S
        s["pool"] = S.PagedCache(*s["cache"])
    return s["pool"]


# ------------------------------------------------------------------------------------------------------ plain, packed

def _padded(x, cu, most):
    """Packed [T, H, D] to [B, H, most, D] in float32; rows past a sequence's end hold another row, masked later."""
    at = (cu[:-1, None].long() + torch.arange(most, device=x.device)[None, :]).clamp(max=x.shape[0] - 1)
    return x[at].transpose(1, 2).float()


def _scores(s):
    """Base-e scores [B, Hkv, g, S, S] of padded causal prompts, -inf where a key is removed, and the rows that are real."""
    cu, most = s["cu"], s["most"]
    B, g = cu.numel() - 1, s["Hq"] // s["Hkv"]
    q = _padded(s["q"], cu, most).reshape(B, s["Hkv"], g * most, s["D"])
    k = _padded(s["k"], cu, most)
    z = torch.matmul(q, k.transpose(2, 3).contiguous()).mul_(1.0 / math.sqrt(s["D"])).view(B, s["Hkv"], g, most, most)
    i = torch.arange(most, device=z.device)
    real = i[None, :] < (cu[1:] - cu[:-1])[:, None]  # [B, S]
    z.masked_fill_(i[None, :] > i[:, None], -math.inf)
    return z, real


def _pack(x, real):
    """Padded [B, H, S, ...] back to packed [T, H, ...]."""
    return x.transpose(1, 2)[real]


def _lse(s):
    z, real = _scores(s)
    B, Hkv, g, S = z.shape[:4]
    m = z.amax(-1)
    return _pack((m + torch.log(z.sub_(m[..., None]).exp_().sum(-1))).view(B, Hkv * g, S), real).contiguous()


def _prompt(s):
    z, real = _scores(s)
    B, Hkv, g, S = z.shape[:4]
    m = z.amax(-1)
    p = z.sub_(m[..., None]).exp_()
    total = p.sum(-1)
    o = torch.matmul(p.view(B, Hkv, g * S, S), _padded(s["v"], s["cu"], s["most"])).view(B, Hkv, g, S, s["D"])
    o = (o / total[..., None]).view(B, Hkv * g, S, s["D"])
    lse = (m + torch.log(total)).view(B, Hkv * g, S)
    return {"o": _pack(o, real).to(s["q"].dtype), "lse": _pack(lse, real)}


def _weights(s):
    z, real = _scores(s)
    B, Hkv, g, S = z.shape[:4]
    lse = _padded(s["lse"][..., None], s["cu"], s["most"]).view(B, Hkv, g, S)
    p = z.sub_(lse[..., None]).exp_()
    p.mul_(real[:, None, None, :, None])
    return {"weights": p.sum((2, 3)) * real[:, None, :]}


# ------------------------------------------------------------------------------------------------------- plain, cache

def _at(codes, *index):
    """Indexed e4m3 codes (as bytes: the same for every build of torch)."""
    return codes.view(torch.uint8)[index].view(E4M3)


def _scale_for(amax):
    """The smallest power of two under which `amax` is at most the largest e4m3 value (2^-126 at least)."""
    f, x = torch.frexp(amax)
    e = torch.where(f <= 0.875, x - 9, x - 8).clamp(min=-126)
    return torch.where(amax > 0, torch.exp2(e.float()), torch.full_like(amax, 2.0 ** -126))


def _append_one(codes, scale, x, s, seq, page, off, tokens_last):
    """Writes the new tokens x [T, H, D] of one of k and v; codes [pages, H, page, D], or [pages, H, D, page]."""
    P, lens, table = s["page"], s["lens"].long(), s["table"].long()
    x = x.float()
    amax = torch.zeros_like(scale).index_reduce_(0, page, x.abs().amax(-1), "amax")
    need = _scale_for(amax)
    new = s["cu"][1:] - s["cu"][:-1]
    tail = table.gather(1, (lens // P).clamp(max=table.shape[1] - 1)[:, None])[:, 0]
    held = (lens % P > 0) & (new > 0)  # sequences that go on in a page they have begun
    was = scale[tail]
    grown = torch.where(held[:, None], torch.maximum(was, need[tail]), need[tail])
    # pages that hold new tokens take the scale these need; begun pages never less than they had
    hit = torch.zeros(scale.shape[0], dtype=torch.bool, device=x.device).index_fill_(0, page, True)
    scale.copy_(torch.where(hit[:, None], need, scale))
    scale[tail] = torch.where((new > 0)[:, None], grown, scale[tail])
    held_codes = _at(codes, tail).float()
    old = held_codes * (was / scale[tail])[..., None, None]
    slot = torch.arange(P, device=x.device)[None, :] < (lens % P)[:, None]
    keep = (slot & held[:, None])[:, None, None, :] if tokens_last else (slot & held[:, None])[:, None, :, None]
    codes.view(torch.uint8)[tail] = torch.where(keep, old, held_codes).to(E4M3).view(torch.uint8)
    y = (x / scale[page][..., None]).clamp(-TOP, TOP).to(E4M3)
    if tokens_last:
        codes.view(torch.uint8).transpose(2, 3)[page, :, off] = y.view(torch.uint8)
    else:
        codes.view(torch.uint8)[page, :, off] = y.view(torch.uint8)


def _append(s):
    k, v, ks, vs = s["cache"]
    T = s["k"].shape[0]
    t = torch.arange(T, device=k.device)
    seq = torch.searchsorted(s["cu"][1:].contiguous(), t.to(torch.int32), right=True)
    pos = s["lens"].long()[seq] + t - s["cu"].long()[seq]
    page, off = s["table"].long()[seq, pos // s["page"]], pos % s["page"]
    _append_one(k, ks, s["k"], s, seq, page, off, False)
    _append_one(v, vs, s["v"], s, seq, page, off, True)
    return {"k": k, "v": v, "k_scale": ks, "v_scale": vs}


def _gathered(s):
    """Keys and values [B, Hkv, L, D] of every page of the table, in float32."""
    k, v, ks, vs = s["cache"]
    at = s["table"].long()
    B, n = at.shape
    kk = (_at(k, at).float() * ks[at][..., None, None]).transpose(1, 2).reshape(B, s["Hkv"], n * s["page"], s["D"])
    vv = (_at(v, at).float() * vs[at][..., None, None]).permute(0, 2, 1, 4, 3).reshape(B, s["Hkv"], n * s["page"], s["D"])
    return kk, vv


def _cache(s):
    k, v = _gathered(s)
    B, Hkv, L, D = k.shape
    g, n = s["Hq"] // Hkv, s["new"]
    q = s["q"].float().view(B, n, Hkv, g, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, g * n, D)
    z = torch.matmul(q, k.transpose(2, 3).contiguous()).view(B, Hkv, g, n, L) * (1.0 / math.sqrt(D))
    last = s["lens"].long()[:, None] - n + torch.arange(n, device=z.device)[None, :]  # the last key a new token sees
    gone = torch.arange(L, device=z.device)[None, None, :] > last[:, :, None]
    z = z.masked_fill(gone[:, None, None], -math.inf)
    m = z.amax(-1, keepdim=True).clamp(min=-1e30)
    p = torch.exp(z - m)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, Hkv, g * n, L), v).view(B, Hkv, g, n, D)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    lse = (m + torch.log(total))[..., 0]
    out = {"o": o.permute(0, 3, 1, 2, 4).reshape(B * n, Hkv * g, D).to(s["q"].dtype),
           "lse": lse.permute(0, 3, 1, 2).reshape(B * n, Hkv * g)}
    if s["weigh"]:
        p = torch.where(total > 0, p / total, torch.zeros_like(p))
        out["weights"] = s["weights_out"].copy_(s["weights"] + p.sum((2, 3))[..., :s["weights"].shape[2]])
    return out


def _evict(s):
    k, v, ks, vs = s["cache"]
    B, Hkv, D, P, budget = len(s["lens"]), s["Hkv"], s["D"], s["page"], s["budget"]
    w, lens = s["weights"], s["lens"].long()[:, None, None]
    j = torch.arange(w.shape[2], device=w.device)
    rank = torch.where(j < lens, torch.where(j >= lens - s["recent"], torch.full_like(w, math.inf), w),
                       torch.full_like(w, -math.inf))
    order = torch.sort(rank, dim=2, descending=True, stable=True).indices
    count = torch.minimum(lens, torch.full_like(lens, budget))  # [B, 1, 1]
    i = torch.arange(min(budget, w.shape[2]), device=w.device)
    kept = torch.where(i < count, order[..., :i.numel()], torch.full_like(order[..., :i.numel()], w.shape[2]))
    kept = kept.sort(2).values
    live = i < count
    kept = torch.where(live, kept, torch.full_like(kept, -1))
    at = kept.clamp(min=0)
    s["weights_out"].zero_()
    s["weights_out"][..., :i.numel()] = torch.where(live, w.gather(2, at), torch.zeros_like(w[..., :1]))
    # tokens to their new pages: pad the kept list to whole pages
    n = s["to"].shape[1]
    full = torch.nn.functional.pad(kept, (0, max(0, n * P - kept.shape[2])), value=-1)[..., :n * P]
    live = (full >= 0).view(B, Hkv, n, P)
    at = full.clamp(min=0)
    page = s["table"].long()[:, None].expand(B, Hkv, -1).gather(2, at // P).view(B, Hkv, n, P)
    off, head = (at % P).view(B, Hkv, n, P), torch.arange(Hkv, device=w.device)[None, :, None, None]
    to = s["to"].long()[:, None].expand(B, Hkv, n)
    used = live.any(3)
    hq = torch.arange(Hkv, device=w.device)[None, :, None].expand(B, Hkv, n)
    for codes, scale, last in ((k, ks, False), (v, vs, True)):
        sc = torch.where(live, scale[page, head], torch.zeros_like(scale[:1, :1]))
        best = sc.amax(3)
        rows = codes.view(torch.uint8).transpose(2, 3)[page, head, off] if last else codes.view(torch.uint8)[page, head, off]
        ratio = torch.where(live, sc / best.clamp(min=2.0 ** -126)[..., None], torch.zeros_like(sc))
        x = (rows.view(E4M3).float() * ratio[..., None]).to(E4M3)
        x = (x.transpose(3, 4) if last else x).contiguous().view(torch.uint8)
        codes.view(torch.uint8)[to[used], hq[used]] = x[used]
        scale[to[used], hq[used]] = best[used]
    kept = torch.nn.functional.pad(kept, (0, budget - kept.shape[2]), value=-1)
    return {"kept": kept.to(torch.int32), "lens": count[:, 0, 0].to(torch.int32), "weights": s["weights_out"],
            "k": k, "v": v, "k_scale": ks, "v_scale": vs}


# ------------------------------------------------------------------------------------------------------------ one pass

def run(state):
    s = state
    if own:
        import sdpa_forward_materialised_amd as S
        if s["op"] == "prompt":
            o, lse = S.prompt_attention(s["q"], s["k"], s["v"], s["cu"], s["cu"], s["most"], s["most"], is_causal=True,
                                        enable_gqa=True)
            return {"o": o, "lse": lse}
        if s["op"] == "weights":
            return {"weights": S.key_weights(s["q"], s["k"], s["lse"], s["cu"], s["cu"], s["most"], s["most"],
                                             is_causal=True, enable_gqa=True)}
        cache = _pool(s)
        if s["op"] == "append":
            S.cache_append(cache, s["k"], s["v"], s["table"], s["lens"], s["cu"], s["most"])
            return {"k": cache.k, "v": cache.v, "k_scale": cache.k_scale, "v_scale": cache.v_scale}
        if s["op"] == "cache":
            w = dict(weights=s["weights"], weights_out=s["weights_out"]) if s["weigh"] else {}
            o, lse = S.cache_attention(s["q"], cache, s["table"], s["lens"], s["cu"], s["new"], s["most_kv"],
                                       enable_gqa=True, **w)
            return {"o": o, "lse": lse, **({"weights": s["weights_out"]} if s["weigh"] else {})}
        kept, lens = S.cache_evict(cache, s["table"], s["lens"], s["weights"], s["budget"], s["recent"], s["to"],
                                   weights_out=s["weights_out"])
        return {"kept": kept, "lens": lens, "weights": s["weights_out"], "k": cache.k, "v": cache.v,
                "k_scale": cache.k_scale, "v_scale": cache.v_scale}
    return {"prompt": _prompt, "weights": _weights, "append": _append, "cache": _cache, "evict": _evict}[s["op"]](s)


# ------------------------------------------------------------------------------------------------------------- exactly

def _round8(x):
    """float64 to the nearest e4m3 value, ties to even, as float64 (x within the range)."""
    _, e = torch.frexp(x)  # x = f 2^e, f in [1/2, 1): the leading bit is 2^(e-1)
    ulp = torch.exp2((e - 1).clamp(min=-6).double() - 3)
    return torch.round(x / ulp) * ulp


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] in ("prompt", "weights"):
        g, cu = c["Hq"] // c["Hkv"], s["cu"].tolist()
        o = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
        lse = torch.empty(s["q"].shape[:2], dtype=torch.float64, device=DEV)
        w = torch.zeros(len(cu) - 1, c["Hkv"], s["most"], dtype=torch.float64, device=DEV)
        for b in range(len(cu) - 1):
            n, rows = cu[b + 1] - cu[b], slice(cu[b], cu[b + 1])
            if n == 0:
                continue
            above = torch.ones(n, n, dtype=torch.bool, device=DEV).triu(1)
            for h in range(c["Hq"]):
                z = s["q"][rows, h].double() @ s["k"][rows, h // g].double().T / math.sqrt(c["D"])
                z.masked_fill_(above, -math.inf)
                if c["op"] == "prompt":
                    lse[rows, h] = torch.logsumexp(z, 1)
                    o[rows, h] = torch.softmax(z, 1) @ s["v"][rows, h // g].double()
                else:
                    w[b, h // g, :n] += torch.exp(z - s["lse"][rows, h].double()[:, None]).sum(0)
                del z
        return {"o": o, "lse": lse} if c["op"] == "prompt" else {"weights": w}
    P, D, Hkv = c["page"], c["D"], c["Hkv"]
    k8, v8, ks, vs = s["cache"]
    lens, table = s["lens"].tolist(), s["table"].long()
    kd, vd = k8.double(), v8.double().transpose(2, 3).contiguous()  # token-major codes
    ks, vs = ks.double(), vs.double()
    if c["op"] == "append":
        cu = s["cu"].tolist()
        for b, n0 in enumerate(lens):
            at = n0
            while at < n0 + cu[b + 1] - cu[b]:
                page, off = int(table[b, at // P]), at % P
                m = min(P - off, n0 + cu[b + 1] - cu[b] - at)
                t = cu[b] + at - n0
                for codes, scale, x in ((kd, ks, s["k"]), (vd, vs, s["v"])):
                    y = x[t:t + m].double().transpose(0, 1)  # [Hkv, m, D]
                    need = torch.exp2(torch.ceil(torch.log2(y.abs().amax((1, 2)) / TOP)))
                    if off:
                        need = torch.maximum(need, scale[page])
                        codes[page, :, :off] = _round8(codes[page, :, :off] * (scale[page] / need)[:, None, None])
                    scale[page] = need
                    codes[page, :, off:off + m] = _round8(y / need[:, None, None])
                at += m
        return {"k": kd, "v": vd.transpose(2, 3).contiguous(), "k_scale": ks, "v_scale": vs}
    if c["op"] == "cache":
        g, n = c["Hq"] // Hkv, c["new"]
        o = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
        lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device=DEV)
        w = s["weights"].double() if c["weigh"] else None
        for b, L in enumerate(lens):
            at = table[b, :-(-L // P)]
            for h in range(Hkv):
                kk = (kd[at, h] * ks[at, h][:, None, None]).reshape(-1, D)[:L]
                vv = (vd[at, h] * vs[at, h][:, None, None]).reshape(-1, D)[:L]
                for i in range(n):
                    see = L - n + i + 1
                    if see <= 0:
                        continue
                    row, heads = b * n + i, slice(h * g, (h + 1) * g)
                    z = s["q"][row, heads].double() @ kk[:see].T / math.sqrt(D)
                    p = torch.softmax(z, 1)
                    lse[row, heads] = torch.logsumexp(z, 1)
                    o[row, heads] = p @ vv[:see]
                    if w is not None:
                        w[b, h, :see] += p.sum(0)
        return {"o": o, "lse": lse, **({"weights": w} if c["weigh"] else {})}
    w, to = s["weights"].double(), s["to"].long()
    wo = torch.zeros_like(w)
    for b, L in enumerate(lens):
        n = min(L, c["budget"])
        for h in range(Hkv):
            late = max(0, L - min(c["recent"], n))
            best = sorted(range(late), key=w[b, h, :late].tolist().__getitem__, reverse=True)[:n - (L - late)]
            keep = torch.tensor(sorted(best) + list(range(late, L)), device=DEV)
            wo[b, h, :n] = w[b, h, keep]
            for codes, scale in ((kd, ks), (vd, vs)):
                page = table[b, keep // P]
                x, sc = codes[page, h, keep % P].clone(), scale[page, h].clone()
                for i in range(-(-n // P)):
                    part = slice(i * P, min(n, i * P + P))
                    top = sc[part].max()
                    whole = torch.zeros(P, D, dtype=torch.float64, device=DEV)
                    whole[:part.stop - part.start] = _round8(x[part] * (sc[part] / top)[:, None])
                    codes[to[b, i], h] = whole
                    scale[to[b, i], h] = top
    return {"kept": None, "lens": None, "weights": wo, "k": kd, "v": vd.transpose(2, 3).contiguous(), "k_scale": ks,
            "v_scale": vs}
