"""The serving operators as a server runs them: prompts, their key weights, the
cache, decode steps and an eviction one after the other; captured into graphs;
on streams of their own; on strided tensors; and on pools past 4 GiB."""

import pytest
import torch

import serving_ref as R
from test_gpu_serving import DEV, TD, _bits, _cu, _fill, _gen, _near

pytestmark = pytest.mark.gpu


def _lib():
    import sdpa_forward_materialised_amd as S
    return S


def _dev(*ts):
    return [t.to(DEV) for t in ts]


def _tokens(g, n, Hq, H, D, dtype):
    q = torch.randn(n, Hq, D, generator=g).to(dtype)
    k, v = (torch.randn(n, H, D, generator=g).to(dtype) for _ in range(2))
    return q, k, v


@pytest.mark.parametrize("dt,D,P,H,Hq", [("bf16", 128, 64, 2, 8), ("f16", 64, 16, 2, 4), ("bf16", 32, 128, 3, 3)])
def test_path(dt, D, P, H, Hq):
    """Prompts -> weights -> cache -> decode -> eviction -> decode, every step against its definition on the CPU."""
    S = _lib()
    g, dtype, gqa = _gen(D + P), TD[dt], Hq != H
    lens = [150, 33, 260]
    B, cap, budget, recent = 3, 320, 96, 24
    pages = -(-cap // P)
    order = torch.randperm(2 * B * pages + 1, generator=g).to(torch.int32)
    table, spare = order[:B * pages].view(B, pages), order[B * pages:2 * B * pages].view(B, pages)
    ref = [t for t in _fill(g, 2 * B * pages + 1, H, P, D)]  # recycled pages: whatever they held
    ref = [ref[0].view(torch.uint8), ref[1].view(torch.uint8), ref[2], ref[3]]
    c = S.PagedCache(*[t.to(DEV).view(torch.float8_e4m3fn) if t.dtype == torch.uint8 else t.to(DEV) for t in ref])
    ref = [t.clone() for t in ref]

    def same_cache(step):
        for name, got, want in zip(("k", "v", "k_scale", "v_scale"), (c.k, c.v, c.k_scale, c.v_scale), ref):
            _bits(f"{step} {name}", got, want)

    # the prompts
    q, k, v = _tokens(g, sum(lens), Hq, H, D, dtype)
    cu = _cu(lens)
    o, lse, to, tl = R.prompt(q, k, v, cu, cu)
    weights = torch.zeros(B, H, cap, device=DEV)
    dq, dk, dv, dcu = _dev(q, k, v, cu)
    O, L = S.prompt_attention(dq, dk, dv, dcu, dcu, max(lens), max(lens), enable_gqa=gqa)
    S.key_weights(dq, dk, L, dcu, dcu, max(lens), max(lens), enable_gqa=gqa, out=weights[:, :, :max(lens)])
    kv = torch.zeros(B, dtype=torch.int32, device=DEV)
    dt_ = table.to(DEV)
    S.cache_append(c, dk, dv, dt_, kv, dcu, max(lens))
    torch.cuda.synchronize()
    _near("prompt O", O, o, to)
    _near("prompt LSE", L, lse, tl)
    w, wt = R.weights(q, k, L.cpu(), cu, cu, max(lens))
    _near("prompt weights", weights[:, :, :max(lens)], w, wt)
    assert (weights[:, :, max(lens):] == 0).all()
    ref = list(R.append([ref[0].view(torch.float8_e4m3fn), ref[1].view(torch.float8_e4m3fn), ref[2], ref[3]], k, v, table,
                        torch.zeros(B, dtype=torch.int32), cu))
    same_cache("prompt")

    def decode(new, kv_lens, tab):
        """new[b] tokens of each sequence, appended and attended; returns the lengths after."""
        nonlocal ref
        q, k, v = _tokens(g, sum(new), Hq, H, D, dtype)
        cu = _cu(new)
        after = kv_lens + torch.tensor(new, dtype=torch.int32)
        w0 = weights.cpu()
        dq, dk, dv, dcu, dl, da, dtab = _dev(q, k, v, cu, kv_lens, after, tab)
        S.cache_append(c, dk, dv, dtab, dl, dcu, max(new))
        O, L = S.cache_attention(dq, c, dtab, da, dcu, max(new), cap, enable_gqa=gqa, weights=weights)
        torch.cuda.synchronize()
        ref = list(R.append([ref[0].view(torch.float8_e4m3fn), ref[1].view(torch.float8_e4m3fn), ref[2], ref[3]], k, v, tab,
                            kv_lens, cu))
        same_cache("decode")
        o, lse, to, tl, wo, tw = R.attention(q, ref, tab, after, cu, w=w0)
        _near("decode O", O, o, to)
        _near("decode LSE", L, lse, tl)
        _near("decode weights", weights, wo, tw)
        return after

    n = torch.tensor(lens, dtype=torch.int32)
    for new in ([1, 1, 1], [1, 1, 1], [4, 1, 3]):
        n = decode(new, n, table)
    # cut to the budget
    w0 = weights.cpu()
    kept, nl = S.cache_evict(c, dt_, n.to(DEV), weights, budget, recent, spare.to(DEV))
    torch.cuda.synchronize()
    rk, rn, rw, *ref = R.evict([ref[0].view(torch.float8_e4m3fn), ref[1].view(torch.float8_e4m3fn), ref[2], ref[3]], table, n,
                               w0, budget, recent, spare)
    _bits("kept", kept, rk)
    _bits("lens", nl, rn)
    assert torch.equal(weights.cpu(), rw)
    same_cache("evict")
    n = nl.cpu()
    for new in ([1, 1, 1], [2, 1, 5], [1, 1, 1]):
        n = decode(new, n, spare)


@pytest.mark.parametrize("new,lens,D,P", [(1, [700, 65, 1], 128, 64), (3, [40, 130, 515], 64, 16)])
def test_decode_step_in_a_graph(new, lens, D, P):
    """append + attention with weights, captured once; five replays with new tokens and lengths, eager work in between."""
    S = _lib()
    g, H, Hq, B, cap = _gen(D), 2, 8, len(lens), 1024
    pages = cap // P
    cache = _fill(g, B * pages, H, P, D)
    table = torch.randperm(B * pages, generator=g).to(torch.int32).view(B, pages).to(DEV)
    a, b = (S.PagedCache(*[t.clone().to(DEV) for t in cache]) for _ in range(2))
    cu = _cu([new] * B).to(DEV)
    q, k, v = (t.to(DEV) for t in _tokens(g, new * B, Hq, H, D, torch.bfloat16))
    before = torch.tensor(lens, dtype=torch.int32, device=DEV)
    after = before + new
    wa = torch.rand(B, H, cap, generator=g).to(DEV)
    wb = wa.clone()
    out = (torch.empty(new * B, Hq, D, dtype=torch.bfloat16, device=DEV), torch.empty(new * B, Hq, device=DEV))

    def step(c, w, o=None):
        S.cache_append(c, k, v, table, before, cu, new)
        return S.cache_attention(q, c, table, after, cu, new, cap, enable_gqa=True, weights=w, out=o)
    step(a, wa, out)  # the first call: nothing is built or sized inside the capture
    step(b, wb)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            step(a, wa, out)
    torch.cuda.current_stream().wait_stream(side)
    for r in range(5):
        q.normal_()
        k.normal_()
        v.normal_()
        before.copy_(after)
        after += new
        graph.replay()
        torch.cuda.synchronize()
        O, L = step(b, wb)
        torch.cuda.synchronize()
        assert torch.equal(O, out[0]) and torch.equal(L, out[1]), f"replay {r}"
        assert torch.equal(wa, wb), f"replay {r}"
        for x, y in ((a.k, b.k), (a.v, b.v), (a.k_scale, b.k_scale), (a.v_scale, b.v_scale)):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8)), f"replay {r}"


def test_prompt_weights_and_eviction_in_a_graph():
    S = _lib()
    g, H, Hq, D, P, B = _gen(77), 2, 4, 64, 32, 2
    lens, budget = [300, 130], 100
    pages = 10
    q, k, v = (t.to(DEV) for t in _tokens(g, sum(lens), Hq, H, D, torch.float16))
    cu = _cu(lens).to(DEV)
    tables = torch.randperm(2 * B * pages, generator=g).to(torch.int32).view(2, B, pages).to(DEV)
    n = torch.tensor(lens, dtype=torch.int32, device=DEV)
    zero = torch.zeros_like(n)
    caches = [S.new_cache(2 * B * pages, H, D, P, DEV) for _ in range(2)]
    ws = [torch.zeros(B, H, 320, device=DEV) for _ in range(2)]

    def run(c, w):
        O, L = S.prompt_attention(q, k, v, cu, cu, 300, 300, enable_gqa=True)
        S.key_weights(q, k, L, cu, cu, 300, 300, enable_gqa=True, out=w[:, :, :300])
        S.cache_append(c, k, v, tables[0], zero, cu, 300)
        kept, nl = S.cache_evict(c, tables[0], n, w, budget, 10, tables[1])
        return O, L, kept, nl
    for c, w in zip(caches, ws):
        run(c, w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            captured = run(caches[0], ws[0])
    torch.cuda.current_stream().wait_stream(side)
    for r in range(4):
        for t in (q, k, v):
            t.normal_()
        graph.replay()
        torch.cuda.synchronize()
        eager = run(caches[1], ws[1])
        torch.cuda.synchronize()
        for x, y in zip(captured, eager):
            assert torch.equal(x, y), f"replay {r}"
        assert torch.equal(ws[0], ws[1])
        assert torch.equal(caches[0].k.view(torch.uint8), caches[1].k.view(torch.uint8))
        assert torch.equal(caches[0].v.view(torch.uint8), caches[1].v.view(torch.uint8))


def test_calls_on_other_streams():
    """Two sequences of calls at once, each on a stream of its own, give the bits of calls one after the other."""
    S = _lib()
    g, H, Hq, D, P, n = _gen(3), 4, 16, 128, 16, 2000
    cache = _fill(g, -(-n // P), H, P, D)
    c = S.PagedCache(*_dev(*cache))
    table = torch.randperm(c.k.shape[0], generator=g).to(torch.int32)[None].to(DEV)
    lens, cu = torch.tensor([n], dtype=torch.int32, device=DEV), _cu([1]).to(DEV)
    qs = [torch.randn(1, Hq, D, generator=g).to(torch.bfloat16).to(DEV) for _ in range(2)]
    pq, pk, pv = _dev(*_tokens(g, 900, Hq, H, D, torch.bfloat16))
    pcu = _cu([900]).to(DEV)

    def calls(q):
        w = torch.zeros(1, H, n, device=DEV)
        r = S.cache_attention(q, c, table, lens, cu, 1, n, enable_gqa=True, weights=w)
        p = S.prompt_attention(pq, pk, pv, pcu, pcu, 900, 900, enable_gqa=True)
        return (*r, w, *p, S.key_weights(pq, pk, p[1], pcu, pcu, 900, 900, enable_gqa=True))
    want = [calls(q) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(calls(qs[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for r in got[i]:
            for x, y in zip(r, want[i]):
                assert torch.equal(x, y)


@pytest.mark.parametrize("dt,D", [("bf16", 128), ("f16", 32), ("f32", 64)])
def test_strided_tensors(dt, D):
    """q, k and v as parts of one projection, the outputs as parts of larger tensors."""
    S = _lib()
    g, H, Hq, n = _gen(D), 2, 6, 170
    qkv = torch.randn(n, Hq + 2 * H, D, generator=g).to(TD[dt])
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + H], qkv[:, Hq + H:]
    cu = _cu([100, 70])
    o, lse, to, tl = R.prompt(q, k, v, cu, cu)
    d = qkv.to(DEV)
    q, k, v = d[:, :Hq], d[:, Hq:Hq + H], d[:, Hq + H:]
    big = torch.full((n, Hq + 1, D + 3), 5.0, dtype=TD[dt], device=DEV)
    stat = torch.full((n, Hq + 2), 5.0, device=DEV)
    O, L = big[:, 1:, 3:], stat[:, :Hq]  # rows of O that take no 16-byte stores
    cu = cu.to(DEV)
    S.prompt_attention(q, k, v, cu, cu, 100, 100, enable_gqa=True, out=(O, L))
    torch.cuda.synchronize()
    _near("O", O, o, to)
    _near("LSE", L, lse, tl)
    assert (big[:, 0] == 5).all() and (big[:, :, :3] == 5).all() and (stat[:, Hq:] == 5).all()
    W, bound = R.weights(qkv[:, :Hq], qkv[:, Hq:Hq + H], L.cpu(), cu.cpu(), cu.cpu(), 100)
    wbig = torch.full((2, H + 1, 120), 5.0, device=DEV)
    S.key_weights(q, k, L, cu, cu, 100, 100, enable_gqa=True, out=wbig[:, :H, 7:107])
    torch.cuda.synchronize()
    _near("weights", wbig[:, :H, 7:107], W, bound)
    assert (wbig[:, H:] == 5).all() and (wbig[:, :, :7] == 5).all() and (wbig[:, :, 107:] == 5).all()
    if dt == "f32":
        return
    # the cache: strided new tokens, queries, outputs and tables
    wide = torch.full((2, 20), -1, dtype=torch.int32, device=DEV)
    wide[:, 5:12] = torch.randperm(14, generator=g).to(torch.int32).view(2, 7).to(DEV)
    table = wide[:, 5:12]
    one, two = S.new_cache(14, H, D, 16, DEV), S.new_cache(14, H, D, 16, DEV)
    zero, lens = torch.zeros(2, dtype=torch.int32, device=DEV), torch.tensor([100, 70], dtype=torch.int32, device=DEV)
    S.cache_append(one, k, v, table, zero, cu, 100)
    S.cache_append(two, k.contiguous(), v.contiguous(), table.contiguous(), zero, cu, 100)
    last = _cu([2, 1]).to(DEV)
    rows = torch.tensor([98, 99, 169], device=DEV)
    ql = torch.full((3, Hq + 2, D), 7.0, dtype=TD[dt], device=DEV)
    ql[:, 1:Hq + 1] = q[rows]
    r1 = S.cache_attention(ql[:, 1:Hq + 1], one, table, lens, last, 2, 100, enable_gqa=True,
                           out=(big[:3, 1:, 3:], stat[:3, :Hq]))
    r2 = S.cache_attention(q[rows], two, table.contiguous(), lens, last, 2, 100, enable_gqa=True)
    torch.cuda.synchronize()
    assert torch.equal(one.k.view(torch.uint8), two.k.view(torch.uint8)) and torch.equal(one.v.view(torch.uint8), two.v.view(torch.uint8))
    assert torch.equal(r1[0], r2[0]) and torch.equal(r1[1], r2[1])


def test_pools_past_4_gib():
    """Pages whose bytes lie past 2^32: the same bits as the same pages in a small pool."""
    S = _lib()
    g, H, Hq, D, P = _gen(11), 8, 16, 128, 128
    far = 40000  # 5.2 GB of k codes, as many of v
    pool = S.PagedCache(torch.empty(far, H, P, D, dtype=torch.float8_e4m3fn, device=DEV),
                        torch.empty(far, H, D, P, dtype=torch.float8_e4m3fn, device=DEV),
                        torch.empty(far, H, device=DEV), torch.empty(far, H, device=DEV))
    small = S.new_cache(8, H, D, P, DEV)
    lens, new = [300, 100], [300, 100]
    q, k, v = _dev(*_tokens(g, 400, Hq, H, D, torch.bfloat16))
    near_t = torch.tensor([[0, 3, 1], [2, 0, 0]], dtype=torch.int32, device=DEV)
    far_t = near_t + far - 8
    to_n = torch.tensor([[4, 5], [6, 7]], dtype=torch.int32, device=DEV)
    cu, zero, n = _cu(new).to(DEV), torch.zeros(2, dtype=torch.int32, device=DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)
    last, rows = _cu([1, 1]).to(DEV), torch.tensor([299, 399], device=DEV)
    got = []
    for c, t, to in ((pool, far_t, to_n + far - 8), (small, near_t, to_n)):
        w = torch.rand(2, H, 300, generator=_gen(5)).to(DEV)
        S.cache_append(c, k, v, t, zero, cu, 300)
        r = S.cache_attention(q[rows], c, t, n, last, 1, 300, enable_gqa=True, weights=w)
        kept, nl = S.cache_evict(c, t, n, w, 130, 20, to)
        r2 = S.cache_attention(q[rows], c, to, nl, last, 1, 130, enable_gqa=True)
        torch.cuda.synchronize()
        whole = t[0, :2].long()  # their tokens fill these pages
        got.append([*r, *r2, w, kept, nl, c.k_scale[whole], c.v_scale[whole], c.k[whole].view(torch.uint8), c.v[whole].view(torch.uint8)])
    for x, y in zip(*got):
        assert torch.equal(x, y)
