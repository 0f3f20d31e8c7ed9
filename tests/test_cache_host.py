"""Host-side checks of the cache in use (no GPU needed): rotary plans against
64-bit angles, and the refusals of every entry point, which enqueue nothing."""
import ctypes
import math

import pytest
import torch

from tests import cache_ref as ref


@pytest.fixture(scope="module")
def lib():
    from decode_kv_cache_02_gb300 import build, rkv
    build.build()
    return rkv.load()


CONFIGS = [dict(rot_dim=64), dict(rot_dim=128, base=500000.0), dict(rot_dim=2),
           dict(rot_dim=96, scaling="linear", factor=4.0),
           dict(rot_dim=128, scaling="ntk", factor=8.0),
           dict(rot_dim=128, scaling="by_parts", factor=8.0, original_len=8192.0, low=1.0, high=4.0),
           dict(rot_dim=64, scaling="by_parts", factor=16.0, original_len=4096.0)]


@pytest.mark.parametrize("cfg", CONFIGS, ids=lambda c: "-".join(str(v) for v in c.values()))
def test_rope_plan_angles(lib, cfg):
    """pos * turns modulo 2^64 is the angle: exact to the plan's rounding of
    f / (2 pi) to 53 bits (and of the power, a few ulp) and to whole units of
    2^-64 (cut off: one unit), both times the position."""
    from decode_kv_cache_02_gb300 import cache
    plan = cache.RopePlan(**cfg)
    f = ref.freqs(cfg["rot_dim"], **{k: v for k, v in cfg.items() if k != "rot_dim"})
    for i, fi in enumerate(f.tolist()):
        turn = fi / (2 * math.pi)
        assert abs(plan._c.turns[i] / 2.0 ** 64 - turn) <= 2.0 ** -50 * turn + 2.0 ** -64
        for pos in (0, 1, -7, 4095, 131071, 2 ** 31 - 1):
            got = ((pos * plan._c.turns[i]) % 2 ** 64) / 2.0 ** 64
            d = (got - pos * turn) % 1.0
            assert min(d, 1 - d) <= abs(pos) * (turn * 2.0 ** -49 + 2.0 ** -64) + 2.0 ** -52


def test_rope_plan_refusals(lib):
    from decode_kv_cache_02_gb300 import cache
    from decode_kv_cache_02_gb300.rkv import RkvError
    for bad in (dict(rot_dim=0), dict(rot_dim=7), dict(rot_dim=130), dict(rot_dim=64, base=0.0),
                dict(rot_dim=64, base=float("nan")), dict(rot_dim=64, factor=0.0),
                dict(rot_dim=2, scaling="ntk", factor=2.0),
                dict(rot_dim=64, scaling="by_parts", factor=2.0, original_len=0.0),
                dict(rot_dim=64, scaling="by_parts", factor=2.0, original_len=10.0, low=4.0, high=4.0),
                dict(rot_dim=64, attn_factor=float("inf")),
                dict(rot_dim=4, freqs=[1.0, float("nan")])):
        with pytest.raises(RkvError) as e:
            cache.RopePlan(**bad)
        assert e.value.code == 1, bad
    with pytest.raises(ValueError):
        cache.RopePlan(64, scaling="other")
    with pytest.raises(ValueError):
        cache.RopePlan(64, freqs=[1.0])
    assert lib.rkv_rope_init(None, None) == 1
    assert lib.rkv_rope_init_freqs(4, 0, None, 1.0, ctypes.byref(cache.RopePlan(4)._c)) == 1
    p = cache.RopePlan(4, freqs=[1.0 + 2 * math.pi, -0.25])  # whole turns drop out; signs stay
    assert abs(p._c.turns[0] / 2.0 ** 64 - 1.0 / (2 * math.pi)) < 2.0 ** -50
    assert abs(p._c.turns[1] / 2.0 ** 64 - (1 - 0.25 / (2 * math.pi))) < 2.0 ** -50


BASE = 1 << 40
GB = 1 << 30


def _rows(off=0, seq=1 << 13, tok=4096, head=128, ptr=None):
    from decode_kv_cache_02_gb300 import rkv
    return bytes(rkv._Rows((BASE + off) if ptr is None else ptr, seq, tok, head))


def _pdesc(**kw):
    from decode_kv_cache_02_gb300 import rkv
    return bytes(rkv._PagedDesc(kw.get("S", 4), kw.get("H", 8), kw.get("G", 4), kw.get("d", 128),
                                kw.get("bs", 16), kw.get("nb", 400), kw.get("mb", 80),
                                kw.get("dtype", 0)))


def test_rope_apply_refusals(lib):
    """Every refused call is answered on the host (made-up addresses)."""
    from decode_kv_cache_02_gb300 import cache
    plan = cache.RopePlan(128)._packed
    some = object()

    def call(plan=plan, dtype=0, d=128, n=10, per=10, pos=BASE, hq=32, q=some, oq=some, hk=8,
             k=some, ok=some):
        q = _rows() if q is some else q
        oq = _rows(GB) if oq is some else oq
        k = _rows(2 * GB) if k is some else k
        ok = _rows(3 * GB) if ok is some else ok
        return lib.rkv_rope_apply(plan, dtype, d, n, per, pos, 0, hq, q, oq, hk, k, ok, None)
    assert call(n=0) == 0                                    # nothing to do
    assert call(plan=None) == 1
    assert call(dtype=2) == 2 and call(d=96) == 2
    assert call(d=64) == 1                                   # rot_dim past the head
    assert call(n=-1) == 1 and call(n=2 ** 31, per=2 ** 31) == 1
    assert call(per=3) == 1 and call(per=0) == 1             # tokens_per_seq does not divide
    assert call(pos=None) == 1 and call(hq=0) == 1 and call(hk=0) == 1
    assert call(hq=20000) == 2
    assert call(q=None) == 1 and call(oq=None) == 1 and call(ok=None) == 1
    assert call(k=None) == 1                                 # out_k without k
    assert call(q=_rows(8)) == 1                             # pointer off 16 bytes
    assert call(q=_rows(tok=4100)) == 1                      # stride off 16 bytes
    assert call(oq=_rows(GB, tok=0)) == 1                    # written rows that meet
    assert call(oq=_rows(GB, head=64)) == 1
    assert call(oq=_rows(128)) == 4                          # output runs into the input
    assert call(ok=_rows(GB + 4096)) == 4                    # the two outputs meet
    assert call(k=_rows(), ok=_rows(), oq=_rows(), q=_rows()) == 4  # one tensor as both, in place
    # in place, rows of a projection: k beginning inside q's heads, or running into the next token
    into = lambda off, tok=6144: dict(q=_rows(tok=tok), oq=_rows(tok=tok), k=_rows(off, tok=tok), ok=_rows(off, tok=tok))  # noqa: E731
    assert call(**into(2 * 31 * 128)) == 4
    assert call(**into(2 * 32 * 128, tok=4096 + 512)) == 4
    assert call(n=0, **into(2 * 32 * 128)) == 0


def test_rows_in_place_of_several_sequences(lib):
    """q and k turned in place, two sequences of five tokens: k between one
    sequence's q and the next, so that one's k is the other's q."""
    from decode_kv_cache_02_gb300 import cache
    plan = cache.RopePlan(128)._packed

    def call(seq, tok):
        q, k = _rows(seq=seq, tok=tok), _rows(2 * 32 * 128, seq=seq, tok=tok)
        return lib.rkv_rope_apply(plan, 0, 128, 10, 5, BASE, 0, 32, q, q, 8, k, k, None)
    assert call(seq=4096, tok=10 * 5120) == 4            # sequences side by side within a token
    assert call(seq=4 * 5120 + 4096, tok=5120) == 4      # the last token's k on the next sequence


def test_append_refusals(lib):
    from decode_kv_cache_02_gb300 import cache, rkv
    some = object()
    q4 = bytes(rkv._Q4Cache(BASE + 10 * GB, BASE + 11 * GB, BASE + 12 * GB, BASE + 13 * GB))

    def call(fn="paged", desc=None, rope=None, K=BASE + 10 * GB, V=BASE + 12 * GB, table=BASE,
             lens=BASE, n=4, new=1, cu=None, pos=None, k=some, v=some, q=some, oq=some, ws=None,
             c=q4):
        desc = _pdesc() if desc is None else desc
        k = _rows() if k is some else k
        v = _rows(GB) if v is some else v
        q = _rows(2 * GB) if q is some else q
        oq = _rows(3 * GB) if oq is some else oq
        if fn == "paged":
            return lib.rkv_paged_append(desc, rope, K, V, table, lens, n, new, cu, pos, k, v, q, oq,
                                        ws, None)
        return lib.rkv_q4_append(desc, rope, c, table, lens, n, new, cu, pos, k, v, q, oq, ws, None)
    for fn in ("paged", "q4"):
        assert call(fn, n=0, new=0) == 0
        assert call(fn, desc=_pdesc(S=0), n=0) == 0
        assert call(fn, n=5) == 1 and call(fn, n=-4, new=-1) == 1   # not new_per_seq each
        assert call(fn, desc=_pdesc(bs=24)) == 1
        assert call(fn, desc=_pdesc(d=256)) == 2 and call(fn, desc=_pdesc(dtype=3)) == 2
        assert call(fn, desc=_pdesc(G=17)) == 2
        assert call(fn, desc=_pdesc(H=2048, G=16)) == 2
        assert call(fn, table=None) == 1 and call(fn, lens=None) == 1
        assert call(fn, k=None) == 1 and call(fn, v=None) == 1
        assert call(fn, oq=None) == 1 and call(fn, q=None) == 1     # q and out_q go together
        assert call(fn, ws=BASE + 16) == 3
        assert call(fn, rope=cache.RopePlan(128)._packed, desc=_pdesc(d=64)) == 1
        assert call(fn, oq=_rows(2 * GB + 256)) == 4                # out_q runs into q
        assert call(fn, q=_rows(), oq=_rows(), k=_rows(2 * 128)) == 4  # q in place over k
        assert call(fn, k=_rows(10 * GB)) == 4                      # input inside the pool
        assert call(fn, oq=_rows(12 * GB)) == 4                     # output inside the pool
    assert call(K=None) == 1 and call(K=BASE + 8) == 1
    assert call(V=BASE + 10 * GB) == 4                              # K and V pools the same
    assert call("q4", c=None) == 1
    assert call("q4", c=bytes(rkv._Q4Cache(BASE, 0, BASE, BASE))) == 1
    assert call("q4", c=bytes(rkv._Q4Cache(BASE + 10 * GB, BASE + 11 * GB, BASE + 10 * GB,
                                           BASE + 13 * GB))) == 4


def test_q4_read_refusals(lib):
    from decode_kv_cache_02_gb300 import rkv
    q4 = bytes(rkv._Q4Cache(BASE + 10 * GB, BASE + 11 * GB, BASE + 12 * GB, BASE + 13 * GB))

    def call(desc=None, c=q4, table=BASE, lens=BASE, n=5, K=BASE + GB, V=BASE + 2 * GB, ws=None):
        return lib.rkv_q4_read(_pdesc() if desc is None else desc, c, table, lens, None, n, K, V,
                               ws, None)
    assert call(n=0) == 0 and call(desc=_pdesc(S=0)) == 0
    assert call(n=-1) == 1 and call(c=None) == 1 and call(table=None) == 1 and call(lens=None) == 1
    assert call(K=None, V=None) == 1 and call(K=BASE + 4) == 1
    assert call(V=BASE + GB + 4096) == 4 and call(K=BASE + 10 * GB) == 4
    assert call(ws=BASE + 8) == 3


def test_attention_sizes_and_refusals(lib):
    from decode_kv_cache_02_gb300 import rkv
    size = lambda T, rows, **kw: lib.rkv_attention_workspace_size(_pdesc(**kw), T, rows)  # noqa: E731
    assert size(1, 100) >= 256
    assert size(0, 100) == 0 and size(1, 0) == 0 and size(1, 80 * 16 + 1) == 0
    assert size(65, 100) == 0 and size(1, 100, d=80) == 0
    # a longer cache never needs less than its own chunks, and an empty batch needs the error word
    assert size(1, 1280, S=0) == 256
    q4 = bytes(rkv._Q4Cache(BASE + 10 * GB, BASE + 11 * GB, BASE + 12 * GB, BASE + 13 * GB))
    some = object()

    def call(fn="paged", desc=None, T=1, q=some, K=BASE + 10 * GB, V=BASE + 12 * GB, c=q4,
             table=BASE, lens=BASE, rows=1280, scale=0.1, out=some, ws=BASE + 20 * GB, n=1 << 40):
        desc = _pdesc() if desc is None else desc
        q = _rows(GB) if q is some else q
        out = _rows(2 * GB) if out is some else out
        if fn == "paged":
            return lib.rkv_paged_attention(desc, T, q, K, V, table, lens, rows, scale, out, None,
                                           ws, n, None)
        return lib.rkv_q4_attention(desc, T, q, c, table, lens, rows, scale, out, None, ws, n, None)
    for fn in ("paged", "q4"):
        assert call(fn, desc=_pdesc(S=0)) == 0
        assert call(fn, T=0) == 1 and call(fn, T=65) == 2
        assert call(fn, rows=0) == 1 and call(fn, rows=1281) == 1
        assert call(fn, scale=float("nan")) == 1 and call(fn, scale=float("inf")) == 1
        assert call(fn, ws=None) == 3 and call(fn, ws=BASE + 128) == 3 and call(fn, n=100) == 3
        assert call(fn, table=None) == 1 and call(fn, lens=None) == 1
        assert call(fn, q=None) == 1 and call(fn, out=None) == 1
        assert call(fn, out=_rows(GB)) == 4                       # out is q
        assert call(fn, out=_rows(12 * GB)) == 4                  # out inside the cache
        assert call(fn, q=_rows(GB + 2)) == 1 and call(fn, q=_rows(GB, head=100)) == 1
        assert call(fn, out=_rows(2 * GB, head=0)) == 1
        assert call(fn, desc=_pdesc(G=32)) == 2
    assert call(K=None) == 1 and call(V=BASE + 2) == 1
    assert call("q4", desc=_pdesc(dtype=1)) == 2                  # 4-bit caches take bf16 queries
    assert call("q4", c=None) == 1


def test_cache_binding_refuses_cpu_tensors(lib):
    from decode_kv_cache_02_gb300 import cache
    q = torch.zeros(2, 1, 4, 64, dtype=torch.bfloat16)
    pool = torch.zeros(4, 2, 8, 64, dtype=torch.bfloat16)
    table, lens = torch.zeros(2, 2, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        cache.rkv_paged_attention(q, pool, pool.clone(), table, lens)
    with pytest.raises(ValueError):
        cache.rkv_paged_append(pool, pool.clone(), q[:, :, :2], q[:, :, :2], table, lens)
    with pytest.raises(ValueError):
        cache.rkv_rope_apply(cache.RopePlan(64), lens, q[:, 0])
    with pytest.raises(ValueError):
        cache.Q4Cache(*([torch.zeros(4, 2, 8, 32, dtype=torch.uint8),
                         torch.zeros(4, 2, 8, 2, 2, dtype=torch.bfloat16)] * 2))


def test_reference_rounds_and_packs():
    """The tests' own 4-bit form: values come back within half a step, the
    ends of a group exactly on the grid's ends."""
    g = torch.Generator().manual_seed(1)
    x = torch.randn(7, 64, generator=g, dtype=torch.float64) * 3 + 1
    c, s, lo = ref.quantise(x)
    back = (c * s[..., None] + lo[..., None]).flatten(-2)
    assert c.min() >= 0 and c.max() <= 15
    assert (back - x).abs().le(s.repeat_interleave(32, -1) * (0.5 + 2.0 ** -20)).all()
    assert torch.equal(lo.to(torch.bfloat16).double(), lo) and torch.equal(s.to(torch.bfloat16).double(), s)
