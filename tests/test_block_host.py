"""Host-side tests of the decoder-layer entries (include/w4a8_block.h): the header, the
binding and the library agree, and bad arguments are refused before the GPU is touched
(every call here fails validation or has nothing to do, so nothing is launched)."""

import ctypes
import os
import re

import pytest

from bit_codebook_quantized_amd import block as B
from bit_codebook_quantized_amd import w4a8

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "w4a8_block.h")
A = 1 << 20          # a 16-byte-aligned fake address (never dereferenced: validation fails first)
OK, INVALID, SHAPE, ALIGN, UNSUPPORTED = range(5)


def declared():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return sorted(set(re.findall(r"^\s*(?:const\s+)?\w+\s*\*?\s*(\w+)\s*\(", text, flags=re.M)))


def test_header_binding_and_library_agree():
    names = declared()
    assert set(names) == set(B.SIGNATURES) and len(names) == 8
    lib = ctypes.CDLL(w4a8.LIB_PATH)
    for n in names:
        assert hasattr(lib, n), n
    assert B.call("w4a8_block_abi_version") == B.ABI_VERSION == 1
    # the structs as a C compiler lays them out
    assert ctypes.sizeof(B.RopeDesc) == 56 and ctypes.sizeof(B.KV8Desc) == 64


def norm(**kw):
    a = dict(x=A, residual=A, stream=0, weight=A, M=2, K=512, eps=1e-6, rot=256, qmax=127, h=A, rstd=A, y=A, xq=A, xs=A)
    assert set(kw) <= set(a)
    return B.call("rmsnorm_quant_act", *(a | kw).values(), None)


def test_norm_validation():
    assert norm(M=0) == OK and norm(M=0, x=None, xq=None, xs=None, y=None, h=None, residual=None) == OK
    assert norm(M=-1) == INVALID and norm(K=-256) == INVALID and norm(M=1 << 22) == SHAPE
    for k in (0, 128, 300):
        assert norm(K=k) == SHAPE
    assert norm(K=16384 + 256) == UNSUPPORTED
    assert norm(stream=2) == INVALID and norm(rot=0) == UNSUPPORTED
    assert norm(qmax=0) == UNSUPPORTED and norm(qmax=128) == UNSUPPORTED
    for e in (0.0, -1.0, float("nan"), float("inf")):
        assert norm(eps=e) == INVALID
    assert norm(x=None) == INVALID and norm(weight=None) == INVALID
    assert norm(xq=None) == INVALID and norm(xs=None) == INVALID and norm(xq=None, xs=None, y=None) == INVALID
    assert norm(residual=None) == INVALID              # an h without a residual
    for p in ("x", "residual", "weight", "h", "y", "xq"):
        assert norm(**{p: A + 8}) == ALIGN, p
    for p in ("rstd", "xs"):
        assert norm(**{p: A + 2}) == ALIGN, p


def grad(**kw):
    a = dict(grad=A, h=A, stream=0, rstd=A, weight=A, grad_h=A, M=2, K=512, rot=256, dx=A, dweight=A, ws=A, size=1 << 30)
    assert set(kw) <= set(a)
    return B.call("rmsnorm_grad", *(a | kw).values(), None)


def test_norm_grad_validation():
    assert grad(M=0, dweight=None) == OK
    assert grad(M=-1) == INVALID and grad(K=100) == SHAPE and grad(K=32768) == UNSUPPORTED and grad(stream=-1) == INVALID
    assert grad(rot=128) == UNSUPPORTED
    for p in ("grad", "h", "rstd", "weight", "dx", "ws"):
        assert grad(**{p: None}) == INVALID, p
    need = B.rmsnorm_grad_workspace(2, 512)
    assert need > 0 and need % (512 * 4) == 0 and grad(size=need - 1) == INVALID
    for p in ("grad", "h", "weight", "grad_h", "dx", "dweight", "ws"):
        assert grad(**{p: A + 4}) == ALIGN, p
    assert B.rmsnorm_grad_workspace(-1, 512) == 0 and B.rmsnorm_grad_workspace(2, 100) == 0
    assert B.rmsnorm_grad_workspace(0, 512) == 0


def rope_desc(**kw):
    a = dict(pos=A, pos_stride=4, inv_freq=A, rotary_dim=64, axes=2, sections=(20, 12), interleaved=0) | kw
    s = (list(a.pop("sections")) + [0] * 4)[:4]
    return B.RopeDesc(a["pos"], a["pos_stride"], a["inv_freq"], a["rotary_dim"], a["axes"], (ctypes.c_int32 * 4)(*s),
                      a["interleaved"])


def rope(desc=None, **kw):
    d = rope_desc() if desc is None else desc
    a = dict(x=A, T=4, heads=3, D=64, xs=192, rope=ctypes.addressof(d), inverse=0, out=A * 2, os=192)
    assert set(kw) <= set(a)
    return B.call("rope_axes", *(a | kw).values(), None)


def test_rope_validation():
    assert rope(T=0, x=None, out=None) == OK
    assert rope(T=-1) == INVALID and rope(heads=0) == INVALID and rope(D=0) == INVALID and rope(inverse=2) == INVALID
    assert rope(D=72, xs=216, os=216) == SHAPE and rope(D=272, xs=816, os=816) == UNSUPPORTED
    assert rope(xs=184) == SHAPE and rope(os=191) == SHAPE and rope(xs=196) == ALIGN
    assert rope(x=None) == INVALID and rope(out=None) == INVALID and rope(x=A + 8) == ALIGN and rope(out=A + 2) == ALIGN
    assert rope(x=A, out=A, xs=200) == INVALID           # in place needs one stride
    assert rope(rope=None) == INVALID
    for bad, st in ((dict(axes=0), INVALID), (dict(axes=5), INVALID), (dict(rotary_dim=80, sections=(20, 20)), SHAPE),
                    (dict(rotary_dim=24, sections=(6, 6)), SHAPE), (dict(sections=(20, 11)), SHAPE),
                    (dict(sections=(40, -8)), INVALID), (dict(pos_stride=3), SHAPE), (dict(pos=None), INVALID),
                    (dict(inv_freq=None), INVALID), (dict(interleaved=2), INVALID), (dict(pos=A + 2), ALIGN)):
        d = rope_desc(**bad)
        assert rope(desc=d) == st, bad


def cache_desc(**kw):
    a = dict(k=A, v=A, k_scale=A, v_scale=A, pages=9, heads=2, head_dim=64, page_tokens=16, table_stride=4, table=A)
    assert set(kw) <= set(a)
    return B.KV8Desc(*(a | kw).values())


BAD_CACHES = ((dict(k=None), INVALID), (dict(v_scale=None), INVALID), (dict(table=None), INVALID), (dict(pages=0), INVALID),
              (dict(heads=0), INVALID), (dict(table_stride=0), INVALID), (dict(head_dim=96), UNSUPPORTED),
              (dict(page_tokens=48), UNSUPPORTED), (dict(page_tokens=256), UNSUPPORTED), (dict(k=A + 8), ALIGN),
              (dict(k_scale=A + 1), ALIGN), (dict(table_stride=1 << 28), SHAPE), (dict(pages=1 << 40), SHAPE))


def append(at=None, desc=None, **kw):
    c = cache_desc() if at is None else at
    r = rope_desc() if desc is None else desc
    a = dict(cache=ctypes.addressof(c), ctx=A, start=A, B=2, T=4, max_new=2, k=A, ks=128, v=A, vs=128, q=A, qh=6, qs=384,
             rope=ctypes.addressof(r), out=A * 2, os=384)
    assert set(kw) <= set(a)
    return B.call("kv8_append", *(a | kw).values(), None)


def test_append_validation():
    assert append(T=0, k=None, v=None) == OK
    for bad, st in BAD_CACHES:
        c = cache_desc(**bad)
        assert append(at=c) == st, bad
    assert append(cache=None) == INVALID
    assert append(B=-1) == INVALID and append(T=-1) == INVALID and append(max_new=-1) == INVALID
    assert append(T=1 << 31) == SHAPE
    for p in ("ctx", "start", "k", "v"):
        assert append(**{p: None}) == INVALID, p
        assert append(**{p: A + 2}) == ALIGN, p
    assert append(q=None) == INVALID and append(out=None) == INVALID and append(qh=0) == INVALID
    assert append(ks=120) == SHAPE and append(vs=132) == ALIGN and append(qs=300) == SHAPE
    assert append(q=A, out=A, qs=400) == INVALID
    d = rope_desc(rotary_dim=80, sections=(20, 20))
    assert append(desc=d) == SHAPE
    assert append(B=1 << 24) == SHAPE                    # more blocks than a launch can have


def attend(cache=None, **kw):
    c = cache_desc() if cache is None else cache
    a = dict(q=A, qh=6, qs=384, cache=ctypes.addressof(c), kv=A, start=A, B=2, T=4, max_new=2, max_kv=50, scale=0.125,
             causal=1, window=0, out=A, os=384, lse=None, ws=None, size=0)
    assert set(kw) <= set(a)
    return B.call("kv8_attention", *(a | kw).values(), None)


def test_attention_validation():
    assert attend(B=0) == OK and attend(T=0, q=None, out=None) == OK and attend(max_new=0) == OK
    for bad, st in BAD_CACHES:
        c = cache_desc(**bad)
        assert attend(cache=c) == st, bad
    for bad in (dict(scale=0.0), dict(scale=-1.0), dict(scale=float("inf")), dict(scale=float("nan")), dict(window=-1),
                dict(causal=2), dict(max_kv=-1), dict(B=-1), dict(T=-1), dict(max_new=-1), dict(q=None), dict(out=None),
                dict(kv=None), dict(start=None), dict(qh=0)):
        assert attend(**bad) == INVALID, bad
    assert attend(qh=5, qs=320, os=320) == SHAPE and attend(qs=320) == SHAPE and attend(os=388) == ALIGN
    assert attend(q=A + 4) == ALIGN and attend(lse=A + 2) == ALIGN
    # a divided context needs its workspace
    need = B.kv8_attention_workspace(2, 4, 2, 60000, 6, 2, 64)
    assert need > 0
    assert attend(max_kv=60000) == INVALID and attend(max_kv=60000, ws=A, size=need - 1) == INVALID
    assert attend(max_kv=60000, ws=A + 4, size=need) == ALIGN
    assert attend(B=1 << 22, T=1 << 22, max_new=4) == SHAPE


def test_workspace_of_sizes_that_are_refused():
    assert B.kv8_attention_workspace(1, 1, 1, 100, 4, 3, 64) == 0
    assert B.kv8_attention_workspace(1, 1, 1, 100, 4, 4, 96) == 0
    assert B.kv8_attention_workspace(-1, 1, 1, 100, 4, 4, 64) == 0


def test_binding_rejects_cpu_tensors():
    import torch
    x = torch.zeros(2, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        B.rmsnorm_quant_act(x, torch.ones(256))
    with pytest.raises(ValueError):
        B.rope_axes(x.view(2, 4, 64), torch.zeros(1, 2, dtype=torch.int32), B.Rope(torch.ones(32)))
    cache = B.KVCache8.empty(2, 1, 64, 16, device="cpu")
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        B.kv8_append(cache, i[None], i, torch.zeros(2, dtype=torch.int32), 1, x.view(8, 1, 64), x.view(8, 1, 64))
    with pytest.raises(ValueError):
        B.kv8_attention(x.view(8, 1, 64), cache, i[None], i, torch.zeros(2, dtype=torch.int32), 1, 1)


def test_attention_counts_the_rows_that_exist():
    """Sizes are bounded by the rows of a batch, not by max_new rows for every sequence."""
    many = dict(B=16384, T=16400, max_new=15, max_kv=60000)      # one sequence of 15 tokens, the others of one
    assert B.kv8_attention_workspace(*many.values(), 128, 32, 64) > 0
    c = cache_desc(heads=32)
    wide = dict(qh=128, qs=8192, os=8192)
    assert attend(cache=c, **many, **wide) == INVALID            # only its workspace is missing
    assert attend(cache=c, **(many | dict(T=1 << 17, max_new=1 << 17)), **wide) == SHAPE     # 2^24 rows
    assert attend(cache=c, **(many | dict(B=1 << 18, T=1 << 13, max_new=60)), **wide) == SHAPE   # 2^24 pairs with a head
    assert attend(cache=c, **(many | dict(B=1 << 30, T=1 << 30, max_new=1 << 30)), **wide) == SHAPE
    assert B.kv8_attention_workspace(1 << 30, 1 << 30, 1 << 30, 1 << 30, 128, 32, 64) == 0


def test_batches_of_no_sequences():
    """An empty table has no address."""
    c = cache_desc(table=None)
    assert attend(cache=c, B=0, kv=None, start=None) == OK and attend(cache=c) == INVALID
    assert append(at=c, B=0, T=0, ctx=None, start=None, k=None, v=None) == OK and append(at=c) == INVALID
