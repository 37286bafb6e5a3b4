"""Key/value cache entry points: what needs no GPU (argument checks that return
before a device is touched, size queries, the rotary frequency table)."""
import ctypes
import math

import pytest
import torch

OK, INVALID, SHAPE, ALIGN, DTYPE, WORKSPACE, CUDA, UNSUP, TIMEOUT = range(9)
FAKE = 1 << 20  # never dereferenced: every call using it fails validation first


@pytest.fixture(scope="module")
def tq():
    from dequant_gemv_tq4_b200 import build as b

    b.build()
    import dequant_gemv_tq4_b200 as tq

    tq.load_library()
    return tq


def _cache(tq, **kw):
    d = dict(codes=FAKE, scales=FAKE, pages=4, page_table=FAKE, batch=2, pages_per_seq=2, page_table_ld=2,
             kv_heads=2, head_dim=64, page_size=16)
    d.update(kw)
    return tq.KvCache(*[d[n] for n, _ in tq.KvCache._fields_])


CACHE_ERRORS = [
    (dict(codes=None), INVALID), (dict(scales=None), INVALID), (dict(page_table=None), INVALID),
    (dict(codes=FAKE + 8), ALIGN), (dict(scales=FAKE + 2), ALIGN), (dict(page_table=FAKE + 2), ALIGN),
    (dict(pages=-1), INVALID), (dict(batch=-1), INVALID), (dict(pages_per_seq=-1), INVALID),
    (dict(page_table_ld=1), INVALID), (dict(kv_heads=0), INVALID), (dict(kv_heads=1025), SHAPE),
    (dict(head_dim=0), INVALID), (dict(head_dim=48), SHAPE), (dict(head_dim=288), SHAPE),
    (dict(page_size=0), INVALID), (dict(page_size=8), SHAPE), (dict(page_size=48), SHAPE),
    (dict(page_size=2048), SHAPE), (dict(batch=4097), SHAPE), (dict(pages=1 << 31), SHAPE),
    (dict(pages_per_seq=(1 << 26) + 1, page_table_ld=1 << 27), SHAPE),
    (dict(batch=512, pages_per_seq=1 << 22, page_table_ld=1 << 22), SHAPE),
]


@pytest.mark.parametrize("kw,want", CACHE_ERRORS)
def test_cache_description_errors(tq, kw, want):
    c = ctypes.byref(_cache(tq, **kw))
    assert tq.tq_kv_append(c, FAKE, FAKE, 3, FAKE, 128, 64, FAKE, 128, 64, 1, None, None, None) == want
    assert tq.tq_kv_read(c, FAKE, FAKE, 3, FAKE, 128, 64, FAKE, 128, 64, 1, None) == want
    assert tq.tq_kv_commit(c, 1, 0, 0, FAKE, FAKE, 4, 4, None) == want
    assert tq.tq_kv_attention(c, FAKE, None, 0, FAKE, 1, 256, 256, 64, FAKE, 1, 256, 256, 64, 1, 4, 1.0, FAKE, 1 << 30,
                              None) == want


def test_append_and_read_argument_errors(tq):
    c = ctypes.byref(_cache(tq))
    rope = tq.RopeDesc(FAKE, 64, 0, 0, 1.0)

    def append(cache=c, seqs=FAKE, places=FAKE, n=3, k=FAKE, kt=128, kh=64, v=FAKE, vt=128, vh=64, t=1, pos=FAKE,
               desc=None):
        return tq.tq_kv_append(cache, seqs, places, n, k, kt, kh, v, vt, vh, t, pos, desc, None)

    assert append(cache=None) == INVALID
    assert append(n=-1) == INVALID
    assert append(n=(1 << 24) + 1) == SHAPE
    assert append(t=3) == DTYPE
    assert append(seqs=None) == INVALID
    assert append(places=None) == INVALID
    assert append(seqs=FAKE + 2) == ALIGN
    assert append(k=None) == INVALID
    assert append(v=None) == INVALID
    assert append(k=FAKE + 8) == ALIGN
    assert append(kt=132) == ALIGN
    assert append(vh=-64) == INVALID
    assert append(n=0) == OK
    assert append(desc=rope, pos=None) == INVALID
    assert append(desc=tq.RopeDesc(None, 64, 0, 0, 1.0)) == INVALID
    assert append(desc=tq.RopeDesc(FAKE, 66, 0, 0, 1.0)) == SHAPE
    assert append(desc=tq.RopeDesc(FAKE, 7, 0, 0, 1.0)) == SHAPE
    assert append(desc=tq.RopeDesc(FAKE, 0, 0, 0, 1.0)) == SHAPE
    assert append(desc=tq.RopeDesc(FAKE, 64, 0, 1, 1.0)) == UNSUP
    assert tq.tq_kv_read(c, FAKE, FAKE, 3, None, 128, 64, FAKE, 128, 64, 1, None) == INVALID
    assert tq.tq_kv_read(c, FAKE, FAKE, 3, FAKE, 128, 60, FAKE, 128, 64, 1, None) == ALIGN
    assert tq.tq_kv_read(c, FAKE, FAKE, 0, FAKE, 128, 64, FAKE, 128, 64, 1, None) == OK


def test_rope_argument_errors(tq):
    desc = tq.RopeDesc(FAKE, 64, 0, 0, 1.0)

    def rope(x=FAKE, out=FAKE, t=1, n=2, heads=3, dim=64, xt=192, xh=64, ot=192, oh=64, pos=FAKE, d=desc):
        return tq.tq_rope(x, out, t, n, heads, dim, xt, xh, ot, oh, pos, d, None)

    assert rope(x=None) == INVALID
    assert rope(out=None) == INVALID
    assert rope(pos=None) == INVALID
    assert rope(d=None) == INVALID
    assert rope(t=4) == DTYPE
    assert rope(n=-1) == INVALID
    assert rope(dim=0) == INVALID
    assert rope(dim=62) == SHAPE
    assert rope(dim=1026) == SHAPE
    assert rope(heads=1025) == SHAPE
    assert rope(x=FAKE + 1) == ALIGN
    assert rope(xt=-1) == INVALID
    # in place with other strides: one element's result would be another's input
    assert rope(xt=256) == INVALID
    assert rope(oh=72) == INVALID
    assert rope(n=0) == OK
    assert rope(heads=0) == OK


def test_attention_argument_errors(tq):
    c = ctypes.byref(_cache(tq))

    def attend(cache=c, lens=FAKE, parents=None, pld=0, q=FAKE, qt=1, qs=(256, 256, 64), out=FAKE, ot=1,
               os=(256, 256, 64), tree=1, heads=4, scale=1.0, ws=FAKE, nbytes=1 << 30):
        return tq.tq_kv_attention(cache, lens, parents, pld, q, qt, *qs, out, ot, *os, tree, heads, scale, ws, nbytes,
                                  None)

    assert attend(heads=3) == SHAPE
    assert attend(heads=0) == INVALID
    assert attend(tree=65) == SHAPE
    assert attend(tree=-1) == INVALID
    assert attend(tree=0) == OK
    assert attend(qt=7) == DTYPE
    assert attend(ot=7) == DTYPE
    assert attend(lens=None) == INVALID
    assert attend(parents=FAKE, pld=3, tree=4) == INVALID
    assert attend(q=None) == INVALID
    assert attend(out=FAKE + 4) == ALIGN
    assert attend(qs=(256, 250, 64)) == ALIGN
    assert attend(qs=(-8, 256, 64)) == INVALID
    assert attend(scale=float("nan")) == INVALID
    assert attend(scale=float("inf")) == INVALID
    assert attend(cache=ctypes.byref(_cache(tq, batch=0))) == OK
    assert attend(cache=ctypes.byref(_cache(tq, pages_per_seq=0, page_table_ld=0))) == SHAPE


def test_commit_argument_errors(tq):
    c = ctypes.byref(_cache(tq))

    def commit(cache=c, layers=2, cs=1 << 16, ss=1 << 14, lens=FAKE, path=FAKE, ld=4, steps=4):
        return tq.tq_kv_commit(cache, layers, cs, ss, lens, path, ld, steps, None)

    assert commit(layers=-1) == INVALID
    assert commit(steps=-1) == INVALID
    assert commit(ld=3) == INVALID
    assert commit(steps=65, ld=65) == SHAPE
    assert commit(cs=8) == ALIGN
    assert commit(ss=4) == ALIGN
    assert commit(cs=-16) == INVALID
    # layers that overlap (a pool here is 8192 bytes of codes, 1024 scales)
    assert commit(cs=0) == INVALID
    assert commit(cs=8192 - 16) == INVALID
    assert commit(ss=1024 - 8) == INVALID
    assert commit(lens=None) == INVALID
    assert commit(path=None) == INVALID
    assert commit(path=FAKE + 1) == ALIGN
    assert commit(layers=0) == OK
    assert commit(steps=0, ld=0) == OK
    assert commit(cache=ctypes.byref(_cache(tq, batch=0))) == OK


def test_size_queries(tq):
    assert tq.tq_kv_codes_bytes(3, 8, 128, 64) == 3 * 2 * 8 * 64 * 64
    assert tq.tq_kv_scales_bytes(3, 8, 128, 64) == 3 * 2 * 8 * 64 * 16
    # 5.0 bits per element
    assert (tq.tq_kv_codes_bytes(5, 2, 96, 16) + tq.tq_kv_scales_bytes(5, 2, 96, 16)) * 8 == 5 * 2 * 2 * 16 * 96 * 5
    for bad in ((-1, 8, 128, 64), (1, 0, 128, 64), (1, 8, 100, 64), (1, 8, 128, 24), (1, 8, 320, 64)):
        assert tq.tq_kv_codes_bytes(*bad) == 0
        assert tq.tq_kv_scales_bytes(*bad) == 0


def test_tensor_helpers_refuse_what_does_not_fit(tq):
    codes = torch.zeros(4, 2, 2, 16, 32, dtype=torch.uint8)
    scales = torch.zeros(4, 2, 2, 16, 4, dtype=torch.int16)
    table = torch.zeros(2, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="codes"):
        tq._cache(codes.to(torch.int8), scales, table)
    with pytest.raises(ValueError, match="scales"):
        tq._cache(codes, scales[..., :2], table)
    with pytest.raises(ValueError, match="page_table"):
        tq._cache(codes, scales, table.long())
    with pytest.raises(ValueError, match="contiguous"):
        tq._cache(codes.transpose(2, 3), scales.transpose(2, 3), table)
    with pytest.raises(ValueError, match="CUDA"):
        tq.rope(torch.zeros(2, 2, 64), torch.zeros(2, dtype=torch.int32), torch.ones(32))
    with pytest.raises(ValueError, match="tokens"):
        tq.rope(torch.zeros(2, 64), torch.zeros(2, dtype=torch.int32), torch.ones(32))
    cpu = torch.device("cpu")
    with pytest.raises(ValueError, match="int32"):
        tq._ints(torch.zeros(3, dtype=torch.int64), "x", cpu, (3,))
    with pytest.raises(ValueError, match="shape"):
        tq._ints(torch.zeros(3, dtype=torch.int32), "x", cpu, (4,))
    with pytest.raises(ValueError, match="unit stride"):
        tq._heads(torch.zeros(2, 4, 8).transpose(1, 2), "x", cpu, (2, 8, 4))


def test_rope_frequencies(tq):
    f = tq.rope_frequencies(64, 10000.0, device="cpu")
    want = [10000.0 ** (-2 * i / 64) for i in range(32)]
    torch.testing.assert_close(f.double(), torch.tensor(want, dtype=torch.float64), rtol=2.0 ** -24, atol=0)
    torch.testing.assert_close(tq.rope_frequencies(64, 10000.0, 4.0, "linear", device="cpu"), f / 4)
    ntk = tq.rope_frequencies(64, 10000.0, 4.0, "ntk", device="cpu")
    assert ntk[0] == 1.0  # the fastest pair stays, the slowest is stretched by exactly the factor
    assert math.isclose(float(ntk[-1]) * 4, float(f[-1]), rel_tol=1e-6)
    parts = tq.rope_frequencies(64, 10000.0, 8.0, "by_parts", original_context=4096, device="cpu")
    turns = 4096 * f.double() / (2 * math.pi)
    assert torch.equal(parts[turns > 4], f[turns > 4])
    torch.testing.assert_close(parts[turns < 1], f[turns < 1] / 8)
    assert torch.all(parts <= f) and torch.all(parts >= f / 8.001)
    for bad in (dict(rot_dim=0), dict(rot_dim=7), dict(rot_dim=8, factor=-1.0), dict(rot_dim=8, scaling="x"),
                dict(rot_dim=2, scaling="ntk"), dict(rot_dim=8, scaling="by_parts", low=4.0)):
        with pytest.raises(ValueError):
            tq.rope_frequencies(device="cpu", **bad)
