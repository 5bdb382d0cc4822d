"""The serving operators' boundary on the CPU: what the C entries and the
binding refuse, before anything is launched, what they accept as empty, and the
workspaces they ask for. No GPU: every call here is refused or has nothing to do."""

import ctypes

import pytest
import torch

import sdpa_forward_materialised_amd as S
from sdpa_forward_materialised_amd import _serving as V

OK, INVALID, UNSUPPORTED = 0, 1, 2
E4 = torch.float8_e4m3fn


def _z(*shape, dtype=torch.float16):
    return torch.zeros(*shape, dtype=dtype)


def _i(*x):
    return torch.tensor(x, dtype=torch.int32)


def _d(t):
    return None if t is None else V._PACK[t.dim()].pack(t.data_ptr() if t.numel() else 0, V._dtype(t), t.dim(), *t.shape, *t.stride())


def _last():
    return S.last_error()


CU = _i(0, 4, 8)


def _prompt(q=None, k=None, v=None, cu_q=CU, cu_k=CU, n=2, mq=4, mk=4, causal=1, scale=0.1, gqa=1, out="q", lse="q"):
    q = _z(8, 4, 64) if q is None else q
    k = _z(8, 2, 64) if k is None else k
    v = _z(8, 2, 64) if v is None else v
    out = torch.empty_like(q) if isinstance(out, str) else out
    lse = _z(*q.shape[:2], dtype=torch.float32) if isinstance(lse, str) else lse
    lib = S.load_library()
    return lib.sdpa_prompt_fwd(_d(q), _d(k), _d(v), cu_q.data_ptr() if cu_q is not None else None,
                               cu_k.data_ptr() if cu_k is not None else None, n, mq, mk, causal, scale, gqa, _d(out),
                               _d(lse), None)


PROMPT_REFUSED = [
    (dict(q=_z(8, 3, 64)), INVALID, "multiple"),
    (dict(gqa=0), INVALID, "enable_gqa"),
    (dict(k=_z(8, 2, 64, dtype=torch.bfloat16)), INVALID, "dtypes differ"),
    (dict(v=_z(8, 2, 64, dtype=torch.float32)), INVALID, "dtypes differ"),
    (dict(k=_z(8, 2, 32)), INVALID, "head dims"),
    (dict(q=_z(8, 4, 48), k=_z(8, 2, 48), v=_z(8, 2, 48)), UNSUPPORTED, "head dim"),
    (dict(v=_z(8, 2, 32)), UNSUPPORTED, "value head dim"),
    (dict(v=_z(7, 2, 64)), INVALID, "tokens or heads"),
    (dict(causal=3), INVALID, "is_causal"),
    (dict(scale=float("nan")), INVALID, "scale"),
    (dict(scale=float("inf")), INVALID, "scale"),
    (dict(n=-1), INVALID, "non-negative"),
    (dict(cu_q=None), INVALID, "cu_seqlens"),
    (dict(out=_z(8, 4, 64, dtype=torch.bfloat16)), INVALID, "query dtype"),
    (dict(out=_z(8, 4, 32)), INVALID, "out dim"),
    (dict(lse=_z(8, 4)), INVALID, "f32"),
    (dict(lse=_z(8, 2, dtype=torch.float32)), INVALID, "lse dim"),
    (dict(q=_z(8, 4, 128)[..., ::2]), UNSUPPORTED, "last dim"),
    (dict(q=_z(8, 4, 65)[..., 1:]), UNSUPPORTED, "aligned"),
    (dict(q=_z(8, 4, 64, dtype=E4)), INVALID, "f32, f16 or bf16"),
]


@pytest.mark.parametrize("change,code,frag", PROMPT_REFUSED, ids=[f"{i}-{c[2]}" for i, c in enumerate(PROMPT_REFUSED)])
def test_prompt_refusals(change, code, frag):
    assert _prompt(**change) == code and frag in _last()


def test_prompt_slice_limit():
    """A (sequence, head) slice of 1 GiB does not fit the kernels' 32-bit extents."""
    big = torch.empty(8, dtype=torch.float16)  # stands for the whole: a refused call touches nothing
    d = V._PACK[3].pack(big.data_ptr(), V._dtype(big), 3, 1 << 20, 2, 64, 1024, 64, 1)
    lib = S.load_library()
    lse = V._PACK[2].pack(big.data_ptr(), 0, 2, 1 << 20, 2, 2, 1)
    m = 1 << 20
    assert lib.sdpa_prompt_fwd(d, d, d, CU.data_ptr(), CU.data_ptr(), 2, m, m, 1, 0.1, 1, d, lse, None) == UNSUPPORTED
    assert "1 GiB" in _last()


def test_absurd_counts_do_not_wrap():
    """Counts whose product leaves 64 bits, on tensors of stride 0, are refused rather than launched."""
    one = torch.empty(64, dtype=torch.float16)
    big = (1 << 31) - 1
    lib = S.load_library()

    def t(rows, heads):
        return V._PACK[3].pack(one.data_ptr(), V._dtype(one), 3, rows, heads, 64, 0, 0, 1)
    lse = V._PACK[2].pack(one.data_ptr(), 0, 2, 1 << 30, big, 0, 1)
    q = t(1 << 30, big)
    assert lib.sdpa_prompt_fwd(q, q, q, CU.data_ptr(), CU.data_ptr(), big, 1 << 30, 1 << 30, 1, 0.1, 0, q, lse,
                               None) == UNSUPPORTED and "grid" in _last()
    q, lse = t(big, 1), V._PACK[2].pack(one.data_ptr(), 0, 2, big, 1, 1, 1)
    assert lib.sdpa_prompt_fwd(q, q, q, CU.data_ptr(), CU.data_ptr(), 2, big, big, 1, 0.1, 0, q, lse,
                               None) == UNSUPPORTED and "2^30" in _last()
    n = ctypes.c_size_t(7)
    assert lib.sdpa_key_weights_workspace_bytes(q, q, 2, 5, big, 0, ctypes.byref(n)) == UNSUPPORTED and n.value == 0


def test_prompt_empty_calls_do_nothing():
    assert _prompt(n=0, cu_q=None, cu_k=None) == OK
    assert _prompt(mq=0) == OK
    assert _prompt(q=_z(0, 4, 64), mq=5) == OK


def _weights(q=None, k=None, lse=None, n=2, mq=4, mk=4, causal=1, scale=0.1, gqa=1, w=None, ws=None, nbytes=0):
    q = _z(8, 4, 64) if q is None else q
    k = _z(8, 2, 64) if k is None else k
    lse = _z(8, 4, dtype=torch.float32) if lse is None else lse
    w = _z(2, 2, 4, dtype=torch.float32) if w is None else w
    return S.load_library().sdpa_key_weights(_d(q), _d(k), _d(lse), CU.data_ptr(), CU.data_ptr(), n, mq, mk, causal, scale,
                                             gqa, _d(w), ws, nbytes, None)


@pytest.mark.parametrize("change,code,frag", [
    (dict(), INVALID, "workspace"),
    (dict(ws=4096 + 8, nbytes=1 << 20), INVALID, "workspace"),
    (dict(ws=4096, nbytes=16), INVALID, "workspace"),
    (dict(w=_z(2, 4, 4, dtype=torch.float32)), INVALID, "weights dim"),
    (dict(w=_z(2, 2, 4)), INVALID, "f32"),
    (dict(w=_z(2, 2, 8, dtype=torch.float32)[..., ::2]), UNSUPPORTED, "last dim"),
    (dict(lse=_z(8, 2, dtype=torch.float32)), INVALID, "lse dim"),
    (dict(gqa=0), INVALID, "enable_gqa"),
    (dict(causal=-1), INVALID, "is_causal"),
])
def test_key_weights_refusals(change, code, frag):
    assert _weights(**change) == code and frag in _last()


def test_key_weights_workspace():
    """Float32 partial sums for every query head of a key head and range of rows."""
    lib, n = S.load_library(), ctypes.c_size_t(7)
    q, k = _d(_z(2000, 4, 64)), _d(_z(2000, 2, 64))
    assert lib.sdpa_key_weights_workspace_bytes(q, k, 3, 1000, 900, 1, ctypes.byref(n)) == OK
    assert n.value % (2 * 3 * 2 * 900 * 4) == 0 and n.value >= 2 * 3 * 2 * 900 * 4
    assert lib.sdpa_key_weights_workspace_bytes(q, k, 3, 1000, 900, 0, ctypes.byref(n)) == INVALID and n.value == 0
    assert lib.sdpa_key_weights_workspace_bytes(q, k, 3, 1000, 0, 1, ctypes.byref(n)) == OK and n.value == 0


def _cache(n=6, H=2, P=16, D=64, k=None, v=None, ks=None, vs=None):
    t = [_z(n, H, P, D, dtype=E4) if k is None else k, _z(n, H, D, P, dtype=E4) if v is None else v,
         _z(n, H, dtype=torch.float32) if ks is None else ks, _z(n, H, dtype=torch.float32) if vs is None else vs]
    return t, b"".join(_d(x) for x in t)


TABLE, LENS = torch.zeros(2, 3, dtype=torch.int32), _i(3, 20)


def _append(cache=None, k=None, v=None, table=TABLE, n=2, pages=3, stride=3, lens=LENS, cu=CU, new=4):
    keep, c = _cache() if cache is None else cache
    k = _z(8, 2, 64) if k is None else k
    v = _z(8, 2, 64) if v is None else v
    p = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    return S.load_library().sdpa_cache_append(c, _d(k), _d(v), p(table), n, pages, stride, p(lens), p(cu), new, None)


CACHE_REFUSED = [
    (dict(P=24), UNSUPPORTED, "pages of 24"),
    (dict(P=256), UNSUPPORTED, "pages of 256"),
    (dict(D=96), UNSUPPORTED, "head dim"),
    (dict(n=0), INVALID, "no pages"),
    (dict(k=_z(6, 2, 16, 64, dtype=torch.float16)), INVALID, "e4m3"),
    (dict(v=_z(6, 2, 16, 64, dtype=E4)), INVALID, "cache v dim"),
    (dict(ks=_z(6, 3, dtype=torch.float32)), INVALID, "k_scale dim"),
    (dict(vs=_z(6, 2, dtype=torch.float16)), INVALID, "f32"),
    (dict(k=_z(6, 2, 64, 16, dtype=E4).transpose(2, 3)), UNSUPPORTED, "last dim"),
    (dict(ks=_z(2, 6, dtype=torch.float32).t()), UNSUPPORTED, "last dim"),
    (dict(v=_z(12, 2, 64, 16, dtype=E4)[::2]), UNSUPPORTED, "contiguous"),
]


@pytest.mark.parametrize("change,code,frag", CACHE_REFUSED, ids=[f"{i}-{c[2]}" for i, c in enumerate(CACHE_REFUSED)])
def test_cache_refusals(change, code, frag):
    assert _append(cache=_cache(**change)) == code and frag in _last()


@pytest.mark.parametrize("change,code,frag", [
    (dict(k=_z(8, 2, 64, dtype=torch.float32)), INVALID, "f16 or bf16"),
    (dict(k=_z(8, 2, 64, dtype=torch.bfloat16)), INVALID, "dtypes differ"),
    (dict(k=_z(8, 4, 64), v=_z(8, 4, 64)), INVALID, "heads"),
    (dict(k=_z(8, 2, 32)), INVALID, "head dim"),
    (dict(v=_z(7, 2, 64)), INVALID, "v dim 0"),
    (dict(k=_z(8, 2, 68)[..., 4:]), UNSUPPORTED, "aligned"),
    (dict(table=None), INVALID, "page_table"),
    (dict(lens=None), INVALID, "kv_lens"),
    (dict(cu=None), INVALID, "cu_seqlens"),
    (dict(stride=2), INVALID, "overlap"),
    (dict(new=-1), INVALID, "max_new"),
    (dict(n=-1), INVALID, "non-negative"),
    (dict(pages=-1), INVALID, "non-negative"),
    (dict(pages=1 << 28), UNSUPPORTED, "2^31"),
    (dict(pages=1 << 62), UNSUPPORTED, "2^31"),
    (dict(pages=(1 << 26) + 1, stride=1 << 27), UNSUPPORTED, "2^30"),
])
def test_append_refusals(change, code, frag):
    assert _append(**change) == code and frag in _last()


def test_append_empty_calls_do_nothing():
    assert _append(new=0) == OK
    assert _append(n=0, table=None, lens=None, cu=None) == OK
    assert _append(k=_z(0, 2, 64), v=_z(0, 2, 64)) == OK


def _attend(q=None, cache=None, mq=4, mkv=48, causal=1, scale=0.1, gqa=1, w=None, wo=None, out="q", lse="q", ws=None,
            nbytes=0, n=2, cu=CU):
    keep, c = _cache() if cache is None else cache
    q = _z(8, 4, 64) if q is None else q
    out = torch.empty_like(q) if isinstance(out, str) else out
    lse = _z(*q.shape[:2], dtype=torch.float32) if isinstance(lse, str) else lse
    return S.load_library().sdpa_cache_attention(_d(q), c, TABLE.data_ptr(), n, 3, 3, LENS.data_ptr(),
                                                 None if cu is None else cu.data_ptr(), mq, mkv, causal, scale, gqa, _d(w),
                                                 _d(wo), _d(out), _d(lse), ws, nbytes, None)


W = _z(2, 2, 48, dtype=torch.float32)
W96 = _z(2, 2, 96, dtype=torch.float32)


@pytest.mark.parametrize("change,code,frag", [
    (dict(q=_z(8, 4, 64, dtype=torch.float32)), INVALID, "f16 or bf16"),
    (dict(q=_z(8, 3, 64)), INVALID, "multiple"),
    (dict(gqa=0), INVALID, "enable_gqa"),
    (dict(q=_z(8, 4, 32)), INVALID, "head dim"),
    (dict(causal=2), INVALID, "is_causal"),
    (dict(mkv=-1), INVALID, "non-negative"),
    (dict(scale=float("inf")), INVALID, "scale"),
    (dict(w=W), INVALID, "together"),
    (dict(wo=W), INVALID, "together"),
    (dict(w=W, wo=W), INVALID, "workspace"),
    (dict(w=_z(2, 4, 48, dtype=torch.float32), wo=W), INVALID, "weights dim"),
    (dict(w=W, wo=_z(2, 2, 40, dtype=torch.float32)), INVALID, "weights_out dim"),
    (dict(w=_z(2, 2, 48), wo=W), INVALID, "f32"),
    (dict(out=_z(8, 4, 32)), INVALID, "out dim"),
    (dict(lse=_z(8, 4)), INVALID, "f32"),
    (dict(cu=None), INVALID, "cu_seqlens_q"),
])
def test_cache_attention_refusals(change, code, frag):
    assert _attend(**change) == code and frag in _last()


def test_cache_attention_empty_calls_do_nothing():
    assert _attend(mq=0) == OK
    assert _attend(q=_z(0, 4, 64)) == OK
    assert _attend(n=0, cu=None) == OK


def test_cache_attention_workspace():
    """None for one range; else statistics and partial outputs for each, and the scores where weights are gathered."""
    lib, n = S.load_library(), ctypes.c_size_t(7)
    keep, c = _cache(D=128)
    q = _d(_z(8, 4, 128))

    def need(mq, mkv, gather, pages=1000):
        assert lib.sdpa_cache_attention_workspace_bytes(q, c, 2, pages, mq, mkv, 1, gather, ctypes.byref(n)) == OK
        return n.value
    assert need(4, 256, 0) == 0
    assert need(4, 16000, 0) > 0 and need(4, 16000, 0) % 4 == 0
    rows = 2 * 2 * 2 * 4
    assert need(4, 256, 1) == 256 + rows * 128 * 4 + rows * 256 * 4  # one range: statistics to 256 bytes, O, scores
    assert need(4, 10 ** 9, 0, pages=10) == need(4, 160, 0, pages=10)  # bounded by the table
    assert lib.sdpa_cache_attention_workspace_bytes(q, c, 2, 10, 4, 100, 0, 0, ctypes.byref(n)) == INVALID and n.value == 0


def _evict(cache=None, w=W, wo=W, budget=16, recent=4, to=TABLE, to_pages=1, stride=1, kept=0, lens=LENS, nl=LENS):
    keep, c = _cache() if cache is None else cache
    p = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    return S.load_library().sdpa_cache_evict(c, TABLE.data_ptr(), 2, 3, 3, p(lens), _d(w), _d(wo), budget, recent, p(to),
                                             to_pages, stride, kept or None, p(nl), None)


@pytest.mark.parametrize("change,code,frag", [
    (dict(budget=0), INVALID, "budget"),
    (dict(budget=1 << 31), INVALID, "budget"),
    (dict(recent=-1), INVALID, "recent"),
    (dict(recent=17), INVALID, "recent"),
    (dict(budget=17, recent=4), INVALID, "need 2"),
    (dict(to_pages=0), INVALID, "need 1"),
    (dict(to_pages=2, stride=1), INVALID, "overlap"),
    (dict(to=None, kept=64), INVALID, "to_table"),
    (dict(kept=0), INVALID, "kept"),
    (dict(nl=None, kept=64), INVALID, "new_lens"),
    (dict(lens=None), INVALID, "kv_lens"),
    (dict(w=_z(2, 2, 48)), INVALID, "f32"),
    (dict(w=_z(2, 3, 48, dtype=torch.float32)), INVALID, "weights dim"),
    (dict(wo=None), INVALID, "weights_out"),
    (dict(budget=(1 << 30) + 1), UNSUPPORTED, "2^30"),
    (dict(kept=64), INVALID, "new_lens overlaps"),
    (dict(kept=64, nl=LENS[1:]), INVALID, "new_lens overlaps"),
    (dict(w=W96[:, :, :48], wo=W96.view(2, 2, 96).as_strided((2, 2, 48), (192, 48, 1)), kept=64), INVALID, "overlap: one"),
])
def test_evict_refusals(change, code, frag):
    assert _evict(**change) == code and frag in _last()


def test_binding_refusals():
    """Every tensor has to be on one GPU; offsets and tables are int32 and contiguous; nothing falls back."""
    q, k = _z(8, 4, 64), _z(8, 2, 64)
    c = S.new_cache(4, 2, 64, 16, "cpu")
    assert c.page_tokens == 16 and c.k.dtype == E4 and c.v.shape == (4, 2, 64, 16)
    with pytest.raises(ValueError, match="GPU only"):
        S.prompt_attention(q, k, k, CU, CU, 4, 4, enable_gqa=True)
    with pytest.raises(ValueError, match="GPU only"):
        S.key_weights(q, k, _z(8, 4, dtype=torch.float32), CU, CU, 4, 4, enable_gqa=True)
    with pytest.raises(ValueError, match="GPU only"):
        S.cache_append(c, k, k, TABLE, LENS, CU, 4)
    with pytest.raises(ValueError, match="GPU only"):
        S.cache_attention(q, c, TABLE, LENS, CU, 4, enable_gqa=True)
    with pytest.raises(ValueError, match="GPU only"):
        S.cache_evict(c, TABLE, LENS, W, 16, 4, TABLE)
    with pytest.raises(AttributeError):  # the C description of the pool would be another's
        c.k = c.k.clone()
    with pytest.raises(ValueError, match="dims"):
        S.PagedCache(c.k[0], c.v, c.k_scale, c.v_scale)
    for bad in (CU.long(), CU[None], torch.zeros(6, dtype=torch.int32)[::2]):
        with pytest.raises(ValueError, match="int32"):
            V._offsets("cu_seqlens", bad)
    with pytest.raises(ValueError, match="entries"):
        V._offsets("kv_lens", CU, 2)
    for bad in (TABLE.long(), TABLE[0], torch.zeros(3, 2, dtype=torch.int32).t()):
        with pytest.raises(ValueError, match="2-D int32"):
            V._table("page_table", bad, 2)
    with pytest.raises(ValueError, match="rows"):
        V._table("page_table", TABLE, 3)
    with pytest.raises(ValueError, match="unsupported dtype"):
        V._desc3("q", torch.zeros(1, 1, 1, dtype=torch.int64))
    with pytest.raises(ValueError, match="3 dims"):
        V._desc3("q", q[0])
