"""Host-side refusals of kvq_map_runs, kvq_append_runs and kvq_attn_runs (no GPU needed: checked before any device work)."""
import ctypes

import pytest

FAKE = 4096  # an aligned address that is never dereferenced
INVALID, LAYOUT = 1, 2


@pytest.fixture(scope="module")
def kvq():
    from quantized_kv_cache_kvq_gb300 import build as b

    b.build()
    import quantized_kv_cache_kvq_gb300 as m

    m.load()
    return m


def cache(kvq, fmt="int8p", **kw):
    d = dict(k_fmt=kvq.FMT[fmt], v_fmt=kvq.FMT[fmt], num_kv_heads=2, num_pages=4, k_data=FAKE, v_data=FAKE, k_scale=FAKE,
             v_scale=FAKE)
    d.update(kw)
    return kvq._Cache(**d)


def test_formats_and_status(kvq):
    for f in kvq.PAGE_SCALED:
        assert [kvq.tile_bytes(f, p) for p in range(8)] == [2048, 2048, 2, 2, 0, 0, 0, 0]
    assert kvq.status_string(9) == "KVQ_ERR_NO_PAGES" and kvq.STATUS[9] == "KVQ_ERR_NO_PAGES"


def test_per_token_entry_points_refuse_page_scaled_caches(kvq):
    L = kvq.lib()
    c = cache(kvq, witness=FAKE)
    assert L.kvq_append(ctypes.byref(c), FAKE, FAKE, 0, FAKE, 1, None, None) == LAYOUT
    assert L.kvq_decode_attn(ctypes.byref(c), None, 0, FAKE, 0, 1, 2, FAKE, 1, FAKE, 1.0, None, FAKE, None, FAKE, 1 << 30,
                             None, None) == LAYOUT


def append(kvq, c, **kw):
    d = dict(k=FAKE, ks=256, v=FAKE, vs=256, dt=1, rs=FAKE, b=1, n=1, bt=FAKE, mp=4, sl=FAKE)
    d.update(kw)
    return kvq.lib().kvq_append_runs(ctypes.byref(c) if c is not None else None, d["k"], d["ks"], d["v"], d["vs"], d["dt"], d["rs"],
                                     d["b"], d["n"], d["bt"], d["mp"], d["sl"], None, None)


def attn(kvq, c, **kw):
    d = dict(q=FAKE, qs=512, dt=1, hq=4, rs=FAKE, b=1, n=1, mr=1, bt=FAKE, mp=4, sl=FAKE, sc=1.0, out=FAKE, lse=None, ws=FAKE,
             wb=1 << 40)
    d.update(kw)
    return kvq.lib().kvq_attn_runs(ctypes.byref(c) if c is not None else None, d["q"], d["qs"], d["dt"], d["hq"], d["rs"], d["b"],
                                   d["n"], d["mr"], d["bt"], d["mp"], d["sl"], d["sc"], d["out"], d["lse"], d["ws"], d["wb"], None,
                                   None)


CACHES = [(dict(num_kv_heads=0), INVALID), (dict(num_kv_heads=129), INVALID), (dict(num_pages=-1), INVALID),
          (dict(reserved=1), INVALID), (dict(reserved2=1), INVALID), (dict(k_data=None), INVALID), (dict(v_data=FAKE + 8), INVALID),
          (dict(k_scale=None), INVALID), (dict(v_scale=FAKE + 2), INVALID), (dict(n_outlier_pairs=2), LAYOUT),
          (dict(k_fmt=3), LAYOUT), (dict(v_fmt=16), LAYOUT), (dict(k_fmt=5, v_fmt=5), LAYOUT)]


@pytest.mark.parametrize("kw,status", CACHES)
def test_cache_refusals(kvq, kw, status):
    c = cache(kvq, **kw)
    assert append(kvq, c) == status
    assert attn(kvq, c) == status


@pytest.mark.parametrize("kw", [
    dict(dt=2), dict(b=-1), dict(b=1025), dict(n=-1), dict(mp=-1), dict(mp=0), dict(rs=None, n=2), dict(ks=255), dict(ks=260),
    dict(vs=128), dict(vs=264 + 4), dict(k=None), dict(v=None), dict(k=FAKE + 8), dict(v=FAKE + 2), dict(sl=None), dict(bt=None)])
def test_append_refusals(kvq, kw):
    assert append(kvq, cache(kvq), **kw) == INVALID
    assert append(kvq, None) == INVALID


@pytest.mark.parametrize("kw,status", [
    (dict(dt=3), INVALID), (dict(hq=3), INVALID), (dict(hq=0), INVALID), (dict(hq=18, qs=18 * 128), LAYOUT), (dict(b=-1), INVALID),
    (dict(b=1025), INVALID), (dict(n=-1), INVALID), (dict(mr=-1), INVALID), (dict(mp=-1), INVALID), (dict(sc=float("inf")), INVALID),
    (dict(sc=float("nan")), INVALID), (dict(rs=None, n=2), INVALID), (dict(rs=None, mr=0), INVALID), (dict(qs=511), INVALID),
    (dict(qs=516), INVALID), (dict(q=None), INVALID), (dict(q=FAKE + 8), INVALID), (dict(out=FAKE + 4), INVALID),
    (dict(out=None), INVALID), (dict(ws=None), INVALID), (dict(ws=FAKE + 8), INVALID), (dict(sl=None), INVALID),
    (dict(bt=None), INVALID), (dict(n=1 << 30, b=2), INVALID)])
def test_attn_refusals(kvq, kw, status):
    assert attn(kvq, cache(kvq), **kw) == status


def test_map_refusals(kvq):
    def call(**kw):
        d = dict(new=FAKE, sl=FAKE, b=2, fp=FAKE, fcap=4, fc=FAKE, bt=FAKE, mp=4, rs=FAKE, slo=FAKE, fco=FAKE, slot=FAKE, pos=FAKE, rows=8)
        d.update(kw)
        return kvq.lib().kvq_map_runs(*d.values(), None, None)

    for kw in (dict(b=-1), dict(b=1025), dict(fcap=-1), dict(mp=-1), dict(rows=-1), dict(new=None), dict(sl=None), dict(fc=None),
               dict(rs=None), dict(slo=None), dict(fco=None), dict(fp=None), dict(bt=None)):
        assert call(**kw) == INVALID, kw


def test_empty_calls_do_nothing(kvq):
    c = cache(kvq)
    assert append(kvq, c, n=0) == 0 and append(kvq, c, b=0) == 0
    assert attn(kvq, c, n=0) == 0 and attn(kvq, c, b=0) == 0
    assert kvq.lib().kvq_attn_runs_workspace_size(1, 1, 1, 2, 3, 1) == 0  # 3 % 2 != 0
    assert kvq.lib().kvq_attn_runs_workspace_size(1025, 1, 1, 2, 4, 1) == 0


def test_host_tensors_are_refused(kvq):
    """Before any pointer reaches the device."""
    import torch

    z = lambda *n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    c = kvq.PagedCache("int8p", "int8p", 1, 4, device="cpu")
    x = torch.zeros((2, 1, 128))
    with pytest.raises(AssertionError):
        kvq.map_runs(z(2), z(2), z(4), z(1), z(2, 2), z(3), z(2), z(1))
    with pytest.raises(AssertionError):
        kvq.append_runs(c, x, x, z(2), z(2, 2))
    with pytest.raises(AssertionError):
        kvq.attn_runs(c, x, z(2), z(2, 2), x.clone(), torch.zeros(4096))
