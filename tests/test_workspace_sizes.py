"""A workspace asked for once, for the largest batch, serves the smaller calls after
it: no GPU needed, sizes and refusals are answered on the host (made-up addresses)."""
import pytest

from tests.test_cache_host import BASE, GB, _pdesc, _rows, lib  # noqa: F401


def needs(lib, kind, S, G, d, dtype, T, rows):  # noqa: F811
    """The least workspace that a call takes, by its refusals of smaller ones: with made-up addresses and no
    table, a call whose workspace is large enough is refused for the table."""
    from decode_kv_cache_02_gb300 import rkv
    desc, q = _pdesc(S=S, H=8, G=G, d=d, dtype=dtype, mb=4096, nb=1 << 20), _rows()
    eight = bytes(rkv._Q8Cache(BASE, BASE + GB, BASE + 2 * GB, BASE + 3 * GB))

    def call(n):
        rest = (None, BASE, rows, 0.1, q, None, BASE, n, None)
        if kind == "paged":
            return lib.rkv_paged_attention(desc, T, q, BASE, BASE, *rest)
        return lib.rkv_q8_attention(desc, T, q, eight, *rest)
    low, high = 0, 1 << 26
    assert call(high) == 1
    while high - low > 1:
        mid = (low + high) // 2
        low, high = (mid, high) if call(mid) == 3 else (low, mid)
    return high


@pytest.mark.parametrize("kind, dtype", [("paged", 0), ("paged", 1), ("q8", 0)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [1, 4, 7, 16])
def test_a_workspace_serves_smaller_calls(lib, kind, dtype, d, G):  # noqa: F811
    """What the size is asked for once, for the largest batch, serves every call with fewer sequences, new tokens or
    rows (a decode loop whose sequences end, drafts of other lengths)."""
    def size(S, T, rows):
        return lib.rkv_attention_workspace_size(_pdesc(S=S, H=8, G=G, d=d, dtype=dtype, mb=4096, nb=1 << 20), T, rows)
    tokens = [1, 2, 3, 4, 5, 6, 7, 8, 9, 12, 13, 16, 17, 24, 25, 32, 33, 48, 49, 63, 64]
    steps = [(S, T, rows) for S in (1, 2, 5, 16, 70) for T in tokens for rows in (64, 65, 200, 9000)]
    need = {x: needs(lib, kind, x[0], G, d, dtype, *x[1:]) for x in steps}
    got = {x: size(*x) for x in steps}
    for x in steps:
        assert all(got[x] >= max(need[y], got[y]) for y in steps if all(a <= b for a, b in zip(y, x))), x
