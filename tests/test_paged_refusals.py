"""The paged cache's entry points refuse bad arguments before any CUDA call
(no GPU needed)."""
import pytest
import torch

from paged_util import Case


@pytest.fixture(scope="module")
def kvq():
    from kv_cache_quantization_02_b200 import kvq
    return kvq


A = 0x7F0000000000          # never dereferenced

BASE = dict(k=A, v=A, dtype=0, k_stride=1024, v_stride=1024, cu=A, start=A, table=A, B=4, max_blocks=64, n=100, Hkv=8,
            D=128, block=64, fmt=0, num_blocks=300, kc=A, vc=A, ks=A, vs=A)


def _write(kvq, **kw):
    a = dict(BASE, **kw)
    return kvq.kvq_paged_write(a["k"], a["v"], a["dtype"], a["k_stride"], a["v_stride"], a["cu"], a["start"],
                               a["table"], a["B"], a["max_blocks"], a["n"], a["Hkv"], a["D"], a["block"], a["fmt"],
                               a["num_blocks"], a["kc"], a["vc"], a["ks"], a["vs"])


def _read(kvq, **kw):
    a = dict(BASE, **kw)
    return kvq.kvq_paged_read(a["cu"], a["start"], a["table"], a["B"], a["max_blocks"], a["n"], a["Hkv"], a["D"],
                              a["block"], a["fmt"], a["num_blocks"], a["kc"], a["vc"], a["ks"], a["vs"], a["dtype"],
                              a["k"], a["v"])


def _attend(kvq, prefill, **kw):
    a = dict(BASE, q=A, q_stride=4096, Hq=32, lens=A, scale=0.1, window=0, out=A, **{})
    a.update(kw)
    head = (a["q"], a["dtype"], a["q_stride"])
    tail = (a["D"], a["block"], a["fmt"], a["num_blocks"], a["kc"], a["vc"], a["ks"], a["vs"], a["scale"],
            a["window"], a["out"])
    if prefill:
        return kvq.kvq_paged_attention_prefill(*head, a["cu"], a["lens"], a["table"], a["B"], a["max_blocks"], a["n"],
                                               a["Hq"], a["Hkv"], *tail)
    return kvq.kvq_paged_attention_decode(*head, a["lens"], a["table"], a["B"], a["max_blocks"], a["Hq"], a["Hkv"],
                                          *tail)


CALLS = [_write, _read, lambda kvq, **kw: _attend(kvq, False, **kw), lambda kvq, **kw: _attend(kvq, True, **kw)]

SHAPES = [
    (dict(D=96), -3), (dict(D=512), -3), (dict(D=0), -3),
    (dict(block=8), -7), (dict(block=48), -7), (dict(block=256), -7), (dict(fmt=2), -7), (dict(fmt=-1), -7),
    (dict(dtype=2), -7), (dict(dtype=-1), -7),
    (dict(B=-1), -5), (dict(max_blocks=-1), -5), (dict(Hkv=0), -5), (dict(num_blocks=-1), -5),
    (dict(num_blocks=1 << 31), -5), (dict(num_blocks=1 << 22), -5), (dict(max_blocks=1 << 26), -5),
]


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("kw,want", SHAPES)
def test_shapes(kvq, call, kw, want):
    assert call(kvq, **kw) == want


@pytest.mark.parametrize("call", CALLS)
def test_null_and_alignment(kvq, call):
    for name in ("kc", "vc", "ks", "vs", "table"):
        assert call(kvq, **{name: 0}) == -1
    for name in ("kc", "vc"):
        assert call(kvq, **{name: A + 8}) == -2
    for name in ("ks", "vs", "table"):
        assert call(kvq, **{name: A + 2}) == -2


def test_nothing_to_do(kvq):
    none = dict(k=0, v=0, cu=0, start=0, table=0, kc=0, vc=0, ks=0, vs=0)
    assert _write(kvq, **none, B=0) == 0 and _write(kvq, **none, n=0) == 0
    assert _read(kvq, **none, B=0) == 0 and _read(kvq, **none, n=0) == 0
    none = dict(none, q=0, lens=0, out=0)
    assert _attend(kvq, False, **none, B=0) == 0
    assert _attend(kvq, True, **none, B=0) == 0 and _attend(kvq, True, **none, n=0) == 0


def test_write_and_read(kvq):
    for call in (_write, _read):
        assert call(kvq, n=-1) == -5 and call(kvq, n=1 << 31) == -5
        assert call(kvq, k=0) == -1 and call(kvq, v=0) == -1 and call(kvq, cu=0) == -1 and call(kvq, start=0) == -1
        assert call(kvq, k=A + 8) == -2 and call(kvq, v=A + 8) == -2
        assert call(kvq, cu=A + 2) == -2 and call(kvq, start=A + 2) == -2
    for name in ("k_stride", "v_stride"):
        for stride in (1020, 1016, 0, -1024, 1028):
            assert _write(kvq, **{name: stride}) == -5
    assert _write(kvq, B=1 << 29, Hkv=1) == -5     # more work items than a grid has


def test_a_scale_beyond_fp32(kvq):
    """The kernels use sm_scale log2(e), which has to be finite too."""
    for prefill in (False, True):
        assert _attend(kvq, prefill, scale=3e38) == -5 and _attend(kvq, prefill, scale=-3e38) == -5


def test_positions_near_two_to_the_31(kvq):
    """Attention rounds positions up to whole key tiles, and a prompt's first query may stand total_q positions before
    the sequence: tables and windows for which that leaves an int are refused (q's alignment is looked at after it)."""
    f = lambda prefill, **kw: _attend(kvq, prefill, q=A + 8, **kw)
    for block in (16, 32, 64, 128):
        most = (2 ** 31 - 1024) // block
        for prefill in (False, True):
            assert f(prefill, block=block, max_blocks=most, num_blocks=9) == -2
            assert f(prefill, block=block, max_blocks=most + 1, num_blocks=9) == -5
        sizes = dict(B=4, Hq=32, Hkv=8, D=128, block=block, window=0)
        assert kvq.kvq_paged_decode_workspace_bytes(max_blocks=most, **sizes) > 0
        assert kvq.kvq_paged_decode_workspace_bytes(max_blocks=most + 1, **sizes) == -1
        assert kvq.kvq_paged_prefill_workspace_bytes(max_blocks=most, total_q=9, **sizes) >= 0
        assert kvq.kvq_paged_prefill_workspace_bytes(max_blocks=most + 1, total_q=9, **sizes) == -1
    wide = dict(max_blocks=(2 ** 31 - 1024) // 64, num_blocks=9, Hq=1, Hkv=1, q_stride=128)
    assert f(True, **wide, n=2 ** 30, window=2 ** 30 - 1) == -2
    assert f(True, **wide, n=2 ** 30, window=2 ** 30) == -5
    assert f(True, **wide, n=2 ** 30, window=2 ** 31 - 1) == -2          # (the whole table: none)
    # the new tokens' write and read have no such rounding
    assert _write(kvq, k=A + 8, max_blocks=(2 ** 31 - 64) // 64, num_blocks=9) == -2
    assert _read(kvq, k=A + 8, max_blocks=(2 ** 31 - 64) // 64, num_blocks=9) == -2


def test_empty_tables_and_caches(kvq):
    """Empty tensors have no address: a table without columns needs none, nor does a cache without blocks (q's or k's
    alignment is looked at after that)."""
    calls = [lambda **kw: _write(kvq, k=A + 8, **kw), lambda **kw: _read(kvq, k=A + 8, **kw),
             lambda **kw: _attend(kvq, False, q=A + 8, **kw), lambda **kw: _attend(kvq, True, q=A + 8, **kw)]
    for f in calls:
        assert f(max_blocks=0, table=0) == -2
        assert f(num_blocks=0, kc=0, vc=0, ks=0, vs=0) == -2
        assert f(max_blocks=0, num_blocks=0, table=0, kc=0, vc=0, ks=0, vs=0) == -2
        assert f(table=0) == -1 and f(kc=0) == -1 and f(vs=0) == -1
        assert f(max_blocks=0, table=0, kc=0) == -1 and f(num_blocks=0, kc=0, vc=0, ks=0, vs=0, table=0) == -1


def test_attention(kvq):
    for prefill in (False, True):
        f = lambda **kw: _attend(kvq, prefill, **kw)
        assert f(Hq=30) == -5 and f(Hq=4) == -5 and f(window=-1) == -5
        assert f(scale=float("inf")) == -5 and f(scale=float("nan")) == -5
        assert f(q_stride=4100) == -5 and f(q_stride=4088) == -5
        for name in ("q", "out", "lens"):
            assert f(**{name: 0}) == -1
        assert f(q=A + 8) == -2 and f(out=A + 8) == -2 and f(lens=A + 2) == -2
    assert _attend(kvq, True, cu=0) == -1 and _attend(kvq, True, cu=A + 2) == -2
    assert _attend(kvq, True, n=-1) == -5 and _attend(kvq, True, n=1 << 31) == -5


def test_workspace_shapes(kvq):
    ok = dict(B=4, max_blocks=64, Hq=32, Hkv=8, D=128, block=64, window=0)
    f = lambda **kw: kvq.kvq_paged_decode_workspace_bytes(**dict(ok, **kw))
    g = lambda **kw: kvq.kvq_paged_prefill_workspace_bytes(**dict(ok, total_q=40, **kw))
    assert f() > 0 and g() >= 0
    assert f(max_blocks=2) == 0 and f(window=100) == 0            # little to split
    for kw in (dict(D=96), dict(block=8), dict(Hq=30), dict(Hkv=0), dict(B=-1), dict(window=-1)):
        assert f(**kw) == -1 and g(**kw) == -1
    assert kvq.kvq_paged_prefill_workspace_bytes(4, 64, -1, 32, 8, 128, 64) == -1
    assert kvq.kvq_status_string(-7).startswith("KVQ_ERR_FORMAT")


def test_what_the_statuses_say(kvq):
    """KVQ_ERR_COUNT is more than the codec's number of vectors: a window, a stride, a softmax scale, ..."""
    text = str(kvq.KvqError(_attend(kvq, False, window=-1)))
    assert text.startswith("KVQ_ERR_COUNT") and "window" in text and "n_vec" in text


def test_binding_checks(kvq):
    """The torch wrappers name the argument that is wrong, before the library is called."""
    c = Case(128, 2, 16, "int8", [3, 4], [5, 6], seed=1)
    k = c.rows(2, "fp16")
    good = [k, k, c.cu, c.start, c.table, *c.cache()]
    with pytest.raises(ValueError, match="CUDA"):
        kvq.paged_write(*good)
    meta = [x.to("meta") for x in good]
    for i, x in ((5, meta[5].to(torch.uint8)), (5, meta[5][0])):
        with pytest.raises(ValueError):
            kvq.paged_write(*[x if j == i else m for j, m in enumerate(meta)])
    with pytest.raises(ValueError):
        kvq.paged_attention_decode(k, c.seq_len, c.table, *c.cache(), sm_scale=1.0)
    with pytest.raises(ValueError):
        kvq.paged_attention_prefill(k, c.cu, c.seq_len, c.table, *c.cache(), sm_scale=1.0)
    with pytest.raises(ValueError):
        kvq.paged_read(c.cu, c.start, c.table, *c.cache(), n_tokens=11)
