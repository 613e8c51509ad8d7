"""The Python binding of the runs' calls on the host: what a cache holds, what is checked before a pointer leaves (CPU)."""
import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def kvq():
    from quantized_kv_cache_kvq_gb300 import build as b

    b.build()
    import quantized_kv_cache_kvq_gb300 as m

    m.load()
    return m


@pytest.mark.parametrize("k_fmt,v_fmt", [("int8p", "int8p"), ("e4m3p", "e4m3p"), ("bf16", "e4m3s"), ("int8", "int8"), ("int8g32", "int8g32")])
def test_bytes_of_a_cache_are_those_of_its_tiles(kvq, k_fmt, v_fmt):
    heads, pages = 3, 5
    c = kvq.PagedCache(k_fmt, v_fmt, heads, pages, device="cpu")
    per_tile = sum(kvq.tile_bytes(f, p) for f, p in ((k_fmt, 0), (v_fmt, 1), (k_fmt, 2), (v_fmt, 3), (k_fmt, 4)))
    assert c.nbytes() == heads * pages * per_tile
