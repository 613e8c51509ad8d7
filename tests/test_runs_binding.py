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


class _Launched(Exception):
    pass


class Elsewhere:
    """A tensor that says it is on device 1."""

    def __init__(self, t):
        self.t = t

    def __getattr__(self, name):
        return (lambda: 1) if name == "get_device" else getattr(self.t, name)


def calls(kvq, monkeypatch, cache):
    """The two calls over ``cache`` on the host; one that gets as far as the launch raises _Launched."""
    def launch(*a):
        raise _Launched

    monkeypatch.setattr(kvq, "_launch", launch)
    # host tensors stand in for the device's: -1 is their device
    x, lens, table = torch.zeros((2, 2, 128)), torch.zeros(2, dtype=torch.int32), torch.zeros((2, 2), dtype=torch.int32)
    return (lambda: kvq.append_runs(cache, x, x, lens, table),
            lambda: kvq.attn_runs(cache, x, lens, table, x.clone(), torch.zeros(64, dtype=torch.uint8)))


PLANES = [("k", lambda t: t[:-1]), ("v", lambda t: t[:-1].clone()), ("v", lambda t: torch.cat([t, t])), ("k", lambda t: t.t()),
          ("k", lambda t: t.float()), ("k", lambda t: torch.cat([t, t], 1)[:, :2048]), ("k_scale", lambda t: t[:, :-1].contiguous()),
          ("v_scale", lambda t: t.t()), ("k_scale", lambda t: t.float()), ("v_scale", lambda t: t[:1])]


@pytest.mark.parametrize("fmt", ["e4m3p", "int8p"])
def test_planes_put_into_a_cache_are_looked_at(kvq, monkeypatch, fmt):
    for name, change in [(None, None), *PLANES]:
        cache = kvq.PagedCache(fmt, fmt, 2, 4, device="cpu")
        for i in range(2):
            with pytest.raises(AssertionError if name else _Launched):
                if name:
                    setattr(cache, name, change(getattr(cache, name)))
                calls(kvq, monkeypatch, cache)[i]()


@pytest.mark.parametrize("name", ["k", "v", "k_scale", "v_scale"])
def test_planes_of_another_device_than_the_calls(kvq, monkeypatch, name):
    cache = kvq.PagedCache("int8p", "int8p", 2, 4, device="cpu")
    setattr(cache, name, Elsewhere(getattr(cache, name)))
    for call in calls(kvq, monkeypatch, cache):
        with pytest.raises(AssertionError):
            call()


def test_a_cache_of_another_format_is_the_librarys_to_refuse(kvq, monkeypatch):
    for call in calls(kvq, monkeypatch, kvq.PagedCache("int8", "int8", 2, 4, device="cpu")):
        with pytest.raises(_Launched):
            call()


@pytest.mark.parametrize("given,starts,passed", [(None, False, 1), (None, True, 6), (3, True, 3), (1, True, 1)])
def test_max_run_is_never_less_than_the_runs_may_be(kvq, monkeypatch, given, starts, passed):
    """Left out, it allows every run that the rows allow: none is skipped unseen."""
    got = []
    monkeypatch.setattr(kvq, "_launch", lambda name, fn, device, stream, *a: got.append(a))
    cache = kvq.PagedCache("int8p", "int8p", 2, 4, device="cpu")
    B = 2 if starts else 6
    lens, table = torch.zeros(B, dtype=torch.int32), torch.zeros((B, 2), dtype=torch.int32)
    q = torch.zeros((6, 4, 128))
    kw = dict(run_starts=torch.zeros(B + 1, dtype=torch.int32)) if starts else {}
    if given is not None:
        kw["max_run"] = given
    kvq.attn_runs(cache, q, lens, table, q.clone(), torch.zeros(64, dtype=torch.uint8), **kw)
    assert got[0][5:8] == (kw["run_starts"].data_ptr() if starts else None, B, 6) and got[0][8] == passed


def test_a_workspace_in_pieces_is_refused(kvq, monkeypatch):
    """Its bytes would be taken in a row from its address, those between the pieces among them."""
    cache = kvq.PagedCache("int8p", "int8p", 2, 4, device="cpu")
    monkeypatch.setattr(kvq, "_launch", lambda *a: None)
    lens, table, q = torch.zeros(2, dtype=torch.int32), torch.zeros((2, 2), dtype=torch.int32), torch.zeros((2, 2, 128))
    ws = torch.zeros((64, 2), dtype=torch.uint8)
    kvq.attn_runs(cache, q, lens, table, q.clone(), ws)
    with pytest.raises(AssertionError):
        kvq.attn_runs(cache, q, lens, table, q.clone(), ws[:, 0])
