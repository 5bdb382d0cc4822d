"""GPU parity of the serving operators (prompt_attention, key_weights, the paged
8-bit cache) against plain float64 definitions, element by element, with the
bounds of serving_ref. Outputs are poisoned with NaN beforehand."""

import pytest
import torch

import serving_ref as R

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TD = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def _lib():
    import sdpa_forward_materialised_amd as S
    return S


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _cu(lens):
    return torch.tensor([0] + list(lens)).cumsum(0).to(torch.int32)


def _near(name, got, want, tol):
    got, want = got.double().cpu(), want.double()
    assert got.shape == want.shape, name
    same = (got == want) | (got.isnan() & want.isnan())
    off = (got - want).abs()
    bad = ~(same | (off <= tol))
    if bad.any():
        i = tuple(int(x) for x in bad.nonzero()[0])
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} off; first at {i}: {got[i]} for {want[i]}, "
                             f"tolerance {tol[i] if torch.is_tensor(tol) else tol}")
    print(f"[result] {name}: worst {float(torch.nan_to_num(off / tol, 0.0, 0.0, 0.0).max() if off.numel() else 0):.3f} of the bound",
          flush=True)


def _packed(seed, lq, lk, Hq, Hkv, D, dtype, spare=0):
    g = _gen(seed)
    q = (1.5 * torch.randn(sum(lq) + spare, Hq, D, generator=g)).to(dtype)
    k = (torch.randn(sum(lk) + spare, Hkv, D, generator=g) + torch.randn(1, Hkv, D, generator=g)).to(dtype)
    v = torch.randn(sum(lk) + spare, Hkv, D, generator=g).to(dtype)
    return q, k, v, _cu(lq), _cu(lk)


def _nan(*shape, dtype=torch.float32):
    return torch.full(shape, float("nan"), dtype=dtype, device=DEV)


# label, seed, query lengths, key lengths, Hq, Hkv, D, dtype, causal, alignment, scale
PROMPTS = [
    ("one-token", 1, [1], [1], 1, 1, 64, "f16", True, "top_left", None),
    ("two-tokens-f32", 2, [2], [2], 2, 2, 32, "f32", True, "top_left", None),
    ("mixed-bf16-d128", 3, [70, 0, 130, 1, 64, 257], [70, 0, 130, 1, 64, 257], 4, 2, 128, "bf16", True, "top_left", None),
    ("mixed-f16-d64", 4, [129, 31, 300], [129, 31, 300], 6, 2, 64, "f16", True, "top_left", None),
    ("long-bf16-d32-gqa7", 5, [700], [700], 7, 1, 32, "bf16", True, "top_left", None),
    ("f32-d128", 6, [65, 100], [65, 100], 2, 1, 128, "f32", True, "top_left", None),
    ("f32-d64-odd", 7, [33, 1, 190], [33, 1, 190], 3, 3, 64, "f32", True, "top_left", None),
    ("f32-long", 21, [700, 3], [700, 3], 2, 2, 64, "f32", True, "top_left", None),
    ("f32-d128-bottom-right", 22, [70, 500], [300, 530], 2, 1, 128, "f32", True, "bottom_right", None),
    ("f32-d32-noncausal", 23, [40, 90], [333, 20], 4, 2, 32, "f32", False, "top_left", None),
    ("f16-d64-blocks", 24, [1, 31, 33, 97, 800], [1, 31, 33, 97, 800], 2, 1, 64, "f16", True, "top_left", None),
    ("bf16-d32-bottom-right", 25, [5, 300, 64], [900, 300, 777], 4, 2, 32, "bf16", True, "bottom_right", None),
    ("f16-d128-noncausal", 26, [33, 129], [800, 95], 2, 1, 128, "f16", False, "top_left", None),
    ("two-groups-d64", 31, [800], [800], 40, 8, 64, "f16", True, "top_left", None),
    ("two-groups-d32", 32, [790, 9], [790, 9], 24, 4, 32, "bf16", True, "top_left", None),
    ("one-group-d64", 33, [300, 70], [300, 70], 48, 6, 64, "bf16", True, "top_left", None),
    ("one-group-d32", 34, [400], [400], 72, 9, 32, "f16", True, "top_left", None),
    ("chunk-bottom-right", 8, [16, 100, 37], [200, 100, 300], 4, 2, 64, "f16", True, "bottom_right", None),
    ("more-queries-than-keys", 9, [90, 40], [30, 0], 2, 2, 128, "bf16", True, "bottom_right", None),
    ("noncausal", 10, [5, 9, 64], [77, 0, 129], 2, 2, 128, "bf16", False, "top_left", None),
    ("negative-scale", 11, [150], [150], 2, 1, 64, "bf16", True, "top_left", -0.3),
    ("zero-scale", 12, [90], [90], 2, 2, 64, "f16", True, "top_left", 0.0),
    ("large-scale", 13, [200], [200], 2, 2, 128, "bf16", True, "top_left", 3.0),
    ("many-heads-8-slices", 14, [64, 200], [64, 200], 8, 8, 64, "bf16", True, "top_left", None),
    ("top-left-longer-keys", 15, [40, 300], [260, 20], 2, 1, 128, "f16", True, "top_left", None),
    ("exact-tiles-bf16", 16, [256, 512], [256, 512], 4, 1, 128, "bf16", True, "top_left", None),
]


@pytest.mark.parametrize("case", PROMPTS, ids=[c[0] for c in PROMPTS])
def test_prompt_and_weights(case):
    S = _lib()
    label, seed, lq, lk, Hq, Hkv, D, dt, causal, align, scale = case
    dtype = TD[dt]
    spare = 3  # tokens behind the last sequence
    q, k, v, cq, ck = _packed(seed, lq, lk, Hq, Hkv, D, dtype, spare)
    o, lse, to, tl = R.prompt(q, k, v, cq, ck, causal, align, scale)
    print(f"[case] prompt {label}", flush=True)
    args = dict(is_causal=causal, scale=scale, enable_gqa=Hq != Hkv, causal_alignment=align)
    dev = [x.to(DEV) for x in (q, k, v, cq, ck)]
    out = (_nan(*q.shape, dtype=dtype), _nan(*q.shape[:2]))
    O, L = S.prompt_attention(*dev, max(lq), max(lk), out=out, **args)
    torch.cuda.synchronize()
    _near(label + " O", O, o, to)
    _near(label + " LSE", L, lse, tl)
    lse32 = torch.nan_to_num(lse, 0.0, float("inf"), -float("inf")).float()
    W, bound = R.weights(q, k, lse32, cq, ck, max(lk), causal, align, scale)
    got = S.key_weights(dev[0], dev[1], lse32.to(DEV), dev[3], dev[4], max(lq), max(lk),
                        out=_nan(len(lq), Hkv, max(lk)), **args)
    torch.cuda.synchronize()
    _near(label + " weights", got, W, bound)


@pytest.mark.parametrize("dt,D,n", [("bf16", 128, 300), ("f16", 64, 130), ("f32", 32, 100), ("bf16", 32, 900),
                                    ("f16", 128, 1000), ("f32", 128, 70), ("f32", 64, 600), ("f16", 64, 1100)])
def test_prompt_values_that_are_not_finite(dt, D, n):
    """NaN and infinities in keys and values reach the rows that keep them, and no other."""
    S = _lib()
    q, k, v, cq, ck = _packed(n + D, [n, 50], [n, 50], 4, 2, D, TD[dt])
    v[n // 2, 0, 3] = float("nan")
    v[n // 3, 1, 5] = float("inf")
    v[n // 3 + 7, 1, 5] = -float("inf")
    v[n - 2, 1, D - 1] = -float("inf")
    v[n + 49, 0, 1] = float("nan")
    k[n - 5, 0, 2] = float("nan")  # its scores are NaN for the rows that keep it
    o, lse, to, tl = R.prompt(q, k, v, cq, ck)
    O, L = S.prompt_attention(*[x.to(DEV) for x in (q, k, v, cq, ck)], n, n, enable_gqa=True)
    torch.cuda.synchronize()
    bad = torch.zeros(n + 50, 4, dtype=torch.bool)
    bad[n - 5:n, :2] = True  # rows of the key head with the NaN key
    assert torch.isnan(L.cpu()[bad]).all() and torch.isnan(O.cpu()[bad]).all()
    _near("O", O.cpu()[~bad], o[~bad], to[~bad])
    _near("LSE", L.cpu()[~bad], lse[~bad], tl[~bad])


def _fill(g, n_pages, H, P, D):
    k = (torch.randn(n_pages, H, P, D, generator=g) * 130).clamp(-448, 448).to(torch.float8_e4m3fn)
    v = (torch.randn(n_pages, H, D, P, generator=g) * 130).clamp(-448, 448).to(torch.float8_e4m3fn)
    ks, vs = (torch.exp2(torch.randint(-9, -4, (n_pages, H), generator=g).float()) for _ in range(2))
    return [k, v, ks, vs]


def _table(g, counts, n_pages, width=None, start=0):
    order = torch.randperm(n_pages, generator=g).to(torch.int32)
    width = max(1, max(counts)) if width is None else width
    t = torch.full((len(counts), width), -7, dtype=torch.int32)  # entries that hold no token are never read
    at = start
    for b, c in enumerate(counts):
        t[b, :c] = order[at:at + c]
        at += c
    assert at <= n_pages
    return t, order


def _bits(name, got, want):
    got = got.cpu()
    got = got.view(torch.uint8) if got.dtype == torch.float8_e4m3fn else got
    d = got != want
    assert not d.any(), f"{name}: {int(d.sum())} of {d.numel()} differ, first at {d.nonzero()[0].tolist()}: " \
                        f"{got[d][0]} for {want[d][0]}"


# label, lengths before, new tokens, Hkv, D, page, dtype, spread of the new tokens' magnitudes
APPENDS = [
    ("first-token", [0], [1], 1, 64, 16, "bf16", 0),
    ("decode", [15, 16, 17, 63, 64, 0], [1, 1, 1, 1, 1, 1], 2, 128, 16, "f16", 0),
    ("prompt", [0, 0, 0], [100, 1, 64], 2, 32, 64, "bf16", 0),
    ("go-on", [5, 130, 16], [200, 3, 0], 3, 64, 32, "f16", 0),
    ("grow", [5, 40, 127], [9, 100, 2], 2, 128, 128, "bf16", 6),
    ("shrink", [5, 40, 127], [9, 100, 2], 2, 32, 128, "bf16", -12),
]


@pytest.mark.parametrize("case", APPENDS, ids=[c[0] for c in APPENDS])
def test_append(case):
    S = _lib()
    label, before, new, H, D, P, dt, spread = case
    g = _gen(len(label) + D)
    counts = [-(-(b + n) // P) for b, n in zip(before, new)]
    n_pages = sum(counts) + 2
    cache = _fill(g, n_pages, H, P, D)
    table, _ = _table(g, counts, n_pages, max(counts) + 1)
    k, v = ((torch.randn(sum(new), H, D, generator=g) * 2.0 ** spread).to(TD[dt]) for _ in range(2))
    lens, cu = torch.tensor(before, dtype=torch.int32), _cu(new)
    want = R.append(cache, k, v, table, lens, cu)
    c = S.PagedCache(*[x.to(DEV) for x in cache])
    print(f"[case] append {label}", flush=True)
    for _ in range(2):  # writing the same tokens again changes nothing
        S.cache_append(c, k.to(DEV), v.to(DEV), table.to(DEV), lens.to(DEV), cu.to(DEV), max(new))
        torch.cuda.synchronize()
        for name, got, ref in zip(("k", "v", "k_scale", "v_scale"), (c.k, c.v, c.k_scale, c.v_scale), want):
            _bits(f"{label} {name}", got, ref)


def test_append_values():
    """Zeros, infinities, NaN, the type's largest and smallest values, ties, tokens past the pages and pages past the pool."""
    S = _lib()
    H, D, P = 2, 32, 16
    g = _gen(5)
    cache = _fill(g, 6, H, P, D)
    table = torch.tensor([[0, 1], [2, 99], [-1, 3], [4, 5]], dtype=torch.int32)
    lens, new = torch.tensor([0, 10, 0, 30], dtype=torch.int32), [16, 12, 20, 9]
    x = torch.randn(sum(new), H, D, generator=g)
    x[0:8] = 0.0
    x[8, 0, 0], x[8, 0, 1], x[8, 0, 2] = float("inf"), -float("inf"), float("nan")
    x[9, 1, :4] = torch.tensor([448.0, 447.0, 440.0, 432.0])
    x[20, 0] = 1e-38
    x[30] = torch.finfo(torch.bfloat16).max
    x = x.to(torch.bfloat16)
    y = x.flip(0).contiguous()
    want = R.append(cache, x, y, table, lens, _cu(new))
    c = S.PagedCache(*[t.to(DEV) for t in cache])
    S.cache_append(c, x.to(DEV), y.to(DEV), table.to(DEV), lens.to(DEV), _cu(new).to(DEV), max(new))
    torch.cuda.synchronize()
    for name, got, ref in zip(("k", "v", "k_scale", "v_scale"), (c.k, c.v, c.k_scale, c.v_scale), want):
        _bits(name, got, ref)


# label, lengths, new tokens, Hq, Hkv, D, page, dtype, causal, weights, max_kv, scale
CACHES = [
    ("one-key", [1], [1], 1, 1, 64, 16, "bf16", True, True, None, None),
    ("decode-f16", [200, 1, 17, 64], [1, 1, 1, 1], 8, 2, 64, 16, "f16", True, False, None, None),
    ("decode-bf16-d128", [300, 513, 128], [1, 1, 1], 8, 2, 128, 64, "bf16", True, True, None, None),
    ("ranges", [1500, 700, 3], [1, 1, 1], 4, 1, 64, 32, "bf16", True, True, None, None),
    ("ranges-no-weights", [2100], [1], 3, 3, 128, 128, "f16", True, False, None, None),
    ("chunks", [90, 33, 700], [8, 3, 5], 8, 2, 128, 32, "bf16", True, True, None, None),
    ("wide-chunk", [100, 61], [30, 61], 7, 1, 32, 16, "f16", True, True, None, None),
    ("empty-and-none", [0, 5, 40], [2, 0, 1], 4, 2, 64, 64, "bf16", True, True, None, None),
    ("chunk-longer-than-cache", [3, 20], [6, 4], 2, 2, 64, 16, "bf16", True, True, None, None),
    ("noncausal", [77, 290], [4, 9], 4, 2, 128, 16, "f16", False, True, None, None),
    ("cut", [400, 90], [1, 2], 4, 2, 64, 64, "bf16", True, True, 130, None),
    ("negative-scale", [150], [3], 4, 2, 64, 64, "bf16", True, True, None, -0.2),
    ("zero-scale", [150], [3], 4, 2, 64, 64, "f16", True, True, None, 0.0),
]


@pytest.mark.parametrize("case", CACHES, ids=[c[0] for c in CACHES])
def test_cache_attention(case):
    S = _lib()
    label, lens, new, Hq, H, D, P, dt, causal, weigh, max_kv, scale = case
    g = _gen(len(label) + sum(lens))
    counts = [-(-n // P) for n in lens]
    cache = _fill(g, sum(counts) + 1, H, P, D)
    table, _ = _table(g, counts, sum(counts) + 1)
    for b, n in enumerate(lens):  # codes past the end may be anything
        if n % P:
            page = int(table[b, n // P])
            cache[0].view(torch.uint8)[page, :, n % P:] = R.NAN8
            cache[1].view(torch.uint8)[page, :, :, n % P:] = R.NAN8
    spare = 2
    q = torch.randn(sum(new) + spare, Hq, D, generator=g).to(TD[dt])
    w = torch.randn(len(lens), H, max(max(lens), 1) + 3, generator=g).abs() if weigh else None
    il, cu = torch.tensor(lens, dtype=torch.int32), _cu(new)
    o, lse, to, tl, wo, tw = R.attention(q, cache, table, il, cu, causal, scale, w, max_kv)
    c = S.PagedCache(*[x.to(DEV) for x in cache])
    out = (_nan(*q.shape, dtype=q.dtype), _nan(*q.shape[:2]))
    print(f"[case] cache {label}", flush=True)
    kw = dict(weights=w.to(DEV), weights_out=_nan(*w.shape)) if weigh else {}
    O, L = S.cache_attention(q.to(DEV), c, table.to(DEV), il.to(DEV), cu.to(DEV), max(new), max_kv, is_causal=causal,
                             scale=scale, enable_gqa=Hq != H, out=out, **kw)
    torch.cuda.synchronize()
    _near(label + " O", O, o, to)
    _near(label + " LSE", L, lse, tl)
    if weigh:
        _near(label + " weights", kw["weights_out"], wo, tw)
        again = w.to(DEV)  # in place gives the same bits
        S.cache_attention(q.to(DEV), c, table.to(DEV), il.to(DEV), cu.to(DEV), max(new), max_kv, is_causal=causal,
                          scale=scale, enable_gqa=Hq != H, weights=again)
        assert torch.equal(again, kw["weights_out"])


@pytest.mark.parametrize("n,D,P,dt", [(8, 128, 64, "bf16"), (5, 64, 16, "f16"), (3, 32, 32, "bf16")])
def test_cache_attention_codes_that_are_not_finite(n, D, P, dt):
    """NaN codes reach the rows that keep their tokens, and no other."""
    S = _lib()
    H, g = 2, _gen(n + D)
    lens, new = [100, 64], [n, n]
    counts = [-(-x // P) for x in lens]
    cache = _fill(g, sum(counts), H, P, D)
    table, _ = _table(g, counts, sum(counts))
    for b, j, h, d in ((0, 99, 0, 3), (0, 98, 1, D - 1), (0, 20, 1, 4), (1, 62, 0, 0)):
        cache[1].view(torch.uint8)[int(table[b, j // P]), h, d, j % P] = R.NAN8 | (128 if d == 4 else 0)
    il, cu = torch.tensor(lens, dtype=torch.int32), _cu(new)
    q = torch.randn(2 * n, 4, D, generator=g).to(TD[dt])
    o, lse, to, tl, _, _ = R.attention(q, cache, table, il, cu)
    c = S.PagedCache(*[x.to(DEV) for x in cache])
    O, L = S.cache_attention(q.to(DEV), c, table.to(DEV), il.to(DEV), cu.to(DEV), n, enable_gqa=True)
    torch.cuda.synchronize()
    assert torch.isnan(o).any() and not torch.isnan(o).all()
    _near("O", O, o, to)
    _near("LSE", L, lse, tl)


def test_cache_attention_pages_past_the_pool():
    """Tokens of a page that is not in the pool are not seen; a row of the table may hold anything past its tokens."""
    S = _lib()
    H, D, P = 2, 64, 16
    g = _gen(9)
    cache = _fill(g, 8, H, P, D)
    table = torch.tensor([[3, 1000, 5, -9], [-1, -1, -1, -1], [7, 2, 1 << 30, 0]], dtype=torch.int32)
    lens, cu = torch.tensor([45, 20, 64], dtype=torch.int32), _cu([1, 2, 3])
    q = torch.randn(6, 4, D, generator=g).to(torch.bfloat16)
    w = torch.zeros(3, H, 64)
    o, lse, to, tl, wo, tw = R.attention(q, cache, table, lens, cu, True, None, w)
    c = S.PagedCache(*[x.to(DEV) for x in cache])
    wd = w.to(DEV)
    O, L = S.cache_attention(q.to(DEV), c, table.to(DEV), lens.to(DEV), cu.to(DEV), 3, enable_gqa=True, weights=wd)
    torch.cuda.synchronize()
    _near("O", O, o, to)
    _near("LSE", L, lse, tl)
    _near("weights", wd, wo, tw)


# label, lengths, Hkv, D, page, budget, recent, what the weights are
EVICTS = [
    ("within-budget", [5, 0, 30], 2, 64, 16, 40, 8, "normal"),
    ("half", [200, 90, 64], 2, 64, 16, 64, 16, "normal"),
    ("odd", [333, 100], 3, 32, 32, 77, 5, "normal"),
    ("no-recent", [150], 1, 128, 64, 33, 0, "normal"),
    ("all-recent", [150, 10], 2, 64, 64, 40, 40, "normal"),
    ("one", [150], 2, 32, 16, 1, 0, "normal"),
    ("ties", [300, 120], 2, 64, 128, 100, 10, "ties"),
    ("equal", [300], 2, 64, 16, 100, 10, "equal"),
    ("signs-and-nan", [300, 200], 2, 32, 16, 90, 10, "odd"),
    ("long", [2500], 1, 32, 128, 600, 100, "ties"),
]


@pytest.mark.parametrize("case", EVICTS, ids=[c[0] for c in EVICTS])
def test_evict(case):
    S = _lib()
    label, lens, H, D, P, budget, recent, kind = case
    g = _gen(len(label) + sum(lens))
    counts, to_counts = [-(-n // P) for n in lens], [-(-min(n, budget) // P) for n in lens]
    n_pages = sum(counts) + sum(to_counts) + 2
    cache = _fill(g, n_pages, H, P, D)
    table, order = _table(g, counts, n_pages)
    to = torch.full((len(lens), -(-budget // P)), -3, dtype=torch.int32)
    at = sum(counts)
    for b, c in enumerate(to_counts):
        to[b, :c] = order[at:at + c]
        at += c
    w = torch.randn(len(lens), H, max(lens) + 5, generator=g)
    if kind == "ties":
        w = (w * 2).round().abs()
    elif kind == "equal":
        w = torch.zeros_like(w)
    elif kind == "odd":
        w = w.round()
        w[:, :, ::7] = -0.0
        w[:, :, 3::31] = float("nan")
        w[:, :, 5::37] = float("inf")
        w[:, :, 9::41] = -float("inf")
    il = torch.tensor(lens, dtype=torch.int32)
    kept, new, wo, kc, vc, ks, vs = R.evict(cache, table, il, w, budget, recent, to)
    c = S.PagedCache(*[x.to(DEV) for x in cache])
    print(f"[case] evict {label}", flush=True)
    w_out = _nan(*w.shape)
    got, nl = S.cache_evict(c, table.to(DEV), il.to(DEV), w.to(DEV), budget, recent, to.to(DEV), weights_out=w_out)
    torch.cuda.synchronize()
    _bits("kept", got, kept)
    _bits("lens", nl, new)
    assert torch.equal(torch.nan_to_num(w_out.cpu(), 7.5), torch.nan_to_num(wo, 7.5))
    for name, x, ref in zip(("k", "v", "k_scale", "v_scale"), (c.k, c.v, c.k_scale, c.v_scale), (kc, vc, ks, vs)):
        _bits(f"{label} {name}", x, ref)
    in_place = w.to(DEV)
    S.cache_evict(c, table.to(DEV), il.to(DEV), in_place, budget, recent, to.to(DEV))
    assert torch.equal(torch.nan_to_num(in_place, 7.5), torch.nan_to_num(w_out, 7.5))


SELECT = [
    # label, lens, budget, recent, weights
    ("close", [6000], 700, 40, lambda g, *s: 1.0 + torch.randint(0, 2000, s, generator=g) * 2.0 ** -23),  # a full bin of the first histogram
    ("two-scales", [9000, 3], 5000, 0, lambda g, *s: torch.where(torch.rand(*s, generator=g) < 0.5, 1e-38, 1.0) * (
        1 + torch.randint(0, 5000, s, generator=g) * 2.0 ** -20)),
    ("many-equal", [12000], 3000, 100, lambda g, *s: torch.randint(0, 3, s, generator=g).float()),
    ("many-recent", [30001], 20000, 19000, lambda g, *s: torch.rand(*s, generator=g)),
    ("recent-only-room", [5000], 4500, 4499, lambda g, *s: torch.rand(*s, generator=g)),
    ("40000", [40000, 17], 4095, 512, lambda g, *s: torch.rand(*s, generator=g).exp2()),
    ("65536", [65536], 65535, 1, lambda g, *s: torch.randn(*s, generator=g)),
    ("denormal", [4097], 64, 0, lambda g, *s: torch.randint(0, 1 << 20, s, generator=g) * 2.0 ** -149),
    ("70000", [70000, 66000, 1], 6000, 300, lambda g, *s: torch.rand(*s, generator=g)),
    ("70000-equal", [70000], 6000, 300, lambda g, *s: torch.ones(*s)),
    ("70000-recent", [70000], 12001, 12000, lambda g, *s: torch.rand(*s, generator=g)),
]


@pytest.mark.parametrize("case", SELECT, ids=[c[0] for c in SELECT])
def test_evict_selection(case):
    """Which tokens stay, and their weights, over many tokens: pages of no pool, so that nothing moves."""
    S = _lib()
    label, lens, budget, recent, draw = case
    B, H, P = len(lens), 2, 128
    w = draw(_gen(sum(lens)), B, H, max(lens) + 3).float()
    pages = -(-max(lens) // P)
    c = S.new_cache(1, H, 32, P, DEV)
    table = torch.full((B, pages), -1, dtype=torch.int32, device=DEV)
    to = torch.full((B, -(-budget // P)), -1, dtype=torch.int32, device=DEV)
    want = torch.full((B, H, budget), -1, dtype=torch.int32)
    wo = torch.zeros_like(w)
    for b, n in enumerate(lens):
        late = max(n - recent, 0) if n > budget else 0
        for h in range(H):
            order = torch.sort(w[b, h, :late], descending=True, stable=True).indices[:budget - (n - late)]
            keep = torch.cat([order.sort().values, torch.arange(late, n)])
            want[b, h, :len(keep)] = keep
            wo[b, h, :len(keep)] = w[b, h, keep]
    il = torch.tensor(lens, dtype=torch.int32).to(DEV)
    print(f"[case] selection {label}", flush=True)
    w_out = _nan(*w.shape)
    kept, nl = S.cache_evict(c, table, il, w.to(DEV), budget, recent, to, weights_out=w_out)
    in_place = w.to(DEV)
    again, _ = S.cache_evict(c, table, il, in_place, budget, recent, to)
    torch.cuda.synchronize()
    _bits("kept", kept, want)
    assert nl.tolist() == [min(n, budget) for n in lens]
    assert torch.equal(w_out.cpu(), wo) and torch.equal(in_place.cpu(), wo)
    assert torch.equal(again, kept)
