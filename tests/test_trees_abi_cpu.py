"""Host-side refusals of the calls for trees of drafted tokens, and what their binding checks (no GPU needed)."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

from tests.test_runs_abi_cpu import CACHES, FAKE, INVALID, LAYOUT, cache, kvq  # noqa: E402, F401


def tree(kvq, **kw):  # noqa: F811
    d = dict(par=FAKE, rs=FAKE, b=2, n=8, sl=FAKE, mask=FAKE, words=1, pos=None)
    d.update(kw)
    return kvq.lib().kvq_tree_runs(*d.values(), None, None)


def rope(kvq, **kw):  # noqa: F811
    d = dict(q=FAKE, qs=512, hq=4, k=FAKE, ks=256, hk=2, dt=1, qw=FAKE, kw=None, eps=1e-6, pos=FAKE, cs=FAKE, mp=10, qo=FAKE, qos=512, ko=FAKE,
             kos=256, rs=FAKE, b=2, n=8)
    d.update(kw)
    return kvq.lib().kvq_rope_runs(*d.values(), None, None)


def attn(kvq, c, **kw):  # noqa: F811
    d = dict(q=FAKE, qs=512, dt=1, hq=4, rs=FAKE, b=1, n=40, mr=40, bt=FAKE, mp=4, sl=FAKE, mask=FAKE, words=2, sc=1.0, out=FAKE, lse=None,
             ws=FAKE, wb=1 << 40)
    d.update(kw)
    return kvq.lib().kvq_attn_tree(ctypes.byref(c) if c is not None else None, *d.values(), None, None)


def verify(kvq, **kw):  # noqa: F811
    d = dict(t=FAKE, ts=100, d=FAKE, ds=100, dt=0, v=100, tok=FAKE, par=FAKE, u=FAKE, rs=FAKE, b=2, n=8, keep=FAKE, kept=FAKE, nxt=FAKE, sl=None,
             slo=None)
    d.update(kw)
    return kvq.lib().kvq_verify_runs(*d.values(), None, None)


def keep(kvq, c, **kw):  # noqa: F811
    d = dict(nc=1, rs=FAKE, b=2, n=8, bt=FAKE, mp=4, sl=FAKE, keep=FAKE, kept=FAKE)
    d.update(kw)
    return kvq.lib().kvq_keep_runs(c, *d.values(), None, None)


@pytest.mark.parametrize("kw", [dict(b=-1), dict(b=1025), dict(n=-1), dict(words=0), dict(rs=None), dict(par=None), dict(sl=None), dict(mask=None)])
def test_tree_refusals(kvq, kw):  # noqa: F811
    assert tree(kvq, **kw) == INVALID


@pytest.mark.parametrize("kw", [
    dict(dt=2), dict(hq=-1), dict(hk=129, ks=129 * 128, kos=129 * 128), dict(hq=1025, qs=1025 * 128, qos=1025 * 128), dict(b=-1), dict(b=1025), dict(n=-1),
    dict(mp=-1), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(q=None), dict(k=None), dict(hq=0), dict(hk=0), dict(pos=None),
    dict(cs=None), dict(cs=FAKE + 4), dict(qo=None), dict(ko=None), dict(q=FAKE + 8), dict(ko=FAKE + 8), dict(qw=FAKE + 4), dict(qs=511), dict(qs=516),
    dict(qos=504), dict(kos=264 + 4), dict(qs=1024)])
def test_rope_refusals(kvq, kw):  # noqa: F811
    assert rope(kvq, **kw) == INVALID


@pytest.mark.parametrize("kw,status", CACHES)
def test_cache_refusals(kvq, kw, status):  # noqa: F811
    c = cache(kvq, **kw)
    assert attn(kvq, c) == status
    assert keep(kvq, ctypes.byref(c)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dt=3), INVALID), (dict(hq=3), INVALID), (dict(hq=18, qs=18 * 128), LAYOUT), (dict(b=-1), INVALID), (dict(b=1025), INVALID), (dict(n=-1), INVALID),
    (dict(mr=-1), INVALID), (dict(mr=1025, words=33), INVALID), (dict(words=1), INVALID), (dict(words=0), INVALID), (dict(words=-1), INVALID),
    (dict(mask=None), INVALID), (dict(sc=float("nan")), INVALID), (dict(rs=None), INVALID), (dict(qs=516), INVALID), (dict(q=None), INVALID),
    (dict(out=FAKE + 4), INVALID), (dict(ws=None), INVALID), (dict(sl=None), INVALID), (dict(bt=None), INVALID)])
def test_attn_refusals(kvq, kw, status):  # noqa: F811
    assert attn(kvq, cache(kvq), **kw) == status
    assert attn(kvq, None) == INVALID


@pytest.mark.parametrize("kw", [
    dict(dt=2), dict(v=0), dict(v=(1 << 19) + 1, ts=1 << 20, ds=1 << 20), dict(b=-1), dict(b=1025), dict(n=-1), dict(rs=None), dict(ts=99), dict(ds=99),
    dict(t=None), dict(tok=None), dict(par=None), dict(keep=None), dict(kept=None), dict(nxt=None), dict(u=None), dict(sl=FAKE), dict(slo=FAKE),
    dict(t=FAKE + 2), dict(d=FAKE + 1), dict(dt=1, t=FAKE + 1)])
def test_verify_refusals(kvq, kw):  # noqa: F811
    assert verify(kvq, **kw) == INVALID


@pytest.mark.parametrize("kw", [dict(nc=-1), dict(b=-1), dict(b=1025), dict(n=-1), dict(mp=-1), dict(mp=0), dict(rs=None), dict(bt=None), dict(sl=None),
                                dict(keep=None), dict(kept=None)])
def test_keep_refusals(kvq, kw):  # noqa: F811
    assert keep(kvq, ctypes.byref(cache(kvq)), **kw) == INVALID
    assert keep(kvq, None) == INVALID


def test_layers_have_to_be_alike(kvq):  # noqa: F811
    two = lambda **kw: (kvq._Cache * 2)(cache(kvq), cache(kvq, **kw))  # noqa: E731
    assert keep(kvq, two(num_pages=5), nc=2) == INVALID
    assert keep(kvq, two(num_kv_heads=1), nc=2) == INVALID
    f = kvq.FMT["e4m3p"]
    assert keep(kvq, two(k_fmt=f, v_fmt=f), nc=2) == LAYOUT
    assert keep(kvq, two(k_scale=None), nc=2) == INVALID


def test_empty_calls_do_nothing(kvq):  # noqa: F811
    c = cache(kvq)
    assert tree(kvq, n=0) == tree(kvq, b=0) == 0
    assert rope(kvq, n=0) == rope(kvq, q=None, hq=0, k=None, hk=0) == 0
    assert attn(kvq, c, n=0) == attn(kvq, c, b=0) == 0
    assert verify(kvq, b=0) == 0
    assert keep(kvq, ctypes.byref(c), n=0) == keep(kvq, ctypes.byref(c), b=0) == keep(kvq, None, nc=0) == 0
    assert kvq.lib().kvq_attn_tree_workspace_size(1, 1, 1, 2, 3, 1) == 0  # 3 % 2 != 0
    assert kvq.lib().kvq_attn_tree_workspace_size(1, 2000, 1025, 2, 4, 1) == 0


# ------------------------------------------------------------------------------------------------ the binding
def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


@pytest.fixture
def sent(kvq, monkeypatch):  # noqa: F811
    """Host tensors stand in for the device's; what would be launched is kept."""
    got = []
    monkeypatch.setattr(kvq, "_launch", lambda name, fn, device, stream, *a: got.append((name, a)))
    return got


def test_host_tensors_are_refused(kvq):  # noqa: F811
    x, c = torch.zeros((2, 1, 128)), kvq.PagedCache("int8p", "int8p", 1, 4, device="cpu")
    for call in (lambda: kvq.tree_runs(i32(2), i32(2), i32(2, 1)), lambda: kvq.rope_runs(x, x, i32(2), torch.zeros(4, 128)),
                 lambda: kvq.attn_tree(c, x, i32(2), i32(2, 2), i32(2, 1), x.clone(), torch.zeros(4096)),
                 lambda: kvq.verify_runs(torch.zeros(2, 5), i32(2), i32(2), None, i32(2), i32(2), i32(2)),
                 lambda: kvq.keep_runs(c, i32(2), i32(2, 2), i32(2), i32(2))):
        with pytest.raises(AssertionError):
            call()


def test_shapes_and_types_are_looked_at(kvq, sent):  # noqa: F811
    x, c = torch.zeros((6, 2, 128)), kvq.PagedCache("int8p", "int8p", 2, 4, device="cpu")
    starts, ws = i32(3), torch.zeros(64, dtype=torch.uint8)
    good = [
        (kvq.tree_runs, dict(parents=i32(6), seq_lens=i32(2), mask=i32(6, 1), positions=i32(6), run_starts=starts),
         dict(parents=i32(5), mask=i32(6, 1).long(), positions=i32(7), run_starts=i32(2), seq_lens=i32(3))),
        (kvq.rope_runs, dict(q=x, k=x, positions=i32(6), cos_sin=torch.zeros(4, 128), q_weight=torch.zeros(128), run_starts=starts),
         dict(k=x.bfloat16(), positions=i32(5), cos_sin=torch.zeros(4, 64), q_weight=torch.zeros(64), q_out=x.bfloat16(), k_out=x[:5], q=x[..., :64])),
        (kvq.attn_tree, dict(cache=c, q=x, seq_lens=i32(2), block_table=i32(2, 2), mask=i32(6, 1), out=x.clone(), workspace=ws, run_starts=starts),
         dict(mask=i32(5, 1), seq_lens=i32(3), out=x[:5], run_starts=i32(2), workspace=torch.zeros(64, 2)[:, 0])),
        (kvq.verify_runs, dict(target=torch.zeros(6, 9), tokens=i32(6), parents=i32(6), uniform=torch.zeros(6, 2), keep=i32(6), kept_lens=i32(2),
                               next_tokens=i32(2), draft=torch.zeros(6, 9), seq_lens=i32(2), seq_lens_out=i32(2), run_starts=starts),
         dict(tokens=i32(5), uniform=torch.zeros(6), draft=torch.zeros(6, 8), keep=i32(5), next_tokens=i32(3), run_starts=None, target=torch.zeros(9, 6).t(),
              seq_lens=i32(3))),
        (kvq.keep_runs, dict(caches=[c, c], seq_lens=i32(2), block_table=i32(2, 2), keep=i32(6), kept_lens=i32(2), run_starts=starts),
         dict(seq_lens=i32(3), kept_lens=i32(1), run_starts=None, keep=i32(6).long())),
    ]
    for fn, kw, changes in good:
        fn(**kw)
        for name, value in changes.items():
            with pytest.raises(AssertionError):
                fn(**dict(kw, **{name: value}))
    assert [name for name, _ in sent] == ["kvq_tree_runs", "kvq_rope_runs", "kvq_attn_tree", "kvq_verify_runs", "kvq_keep_runs"]


@pytest.mark.parametrize("given,starts,words,passed", [(None, False, 1, 1), (None, True, 3, 70), (None, True, 2, 64), (7, True, 2, 7)])
def test_max_run_is_never_less_than_the_runs_may_be(kvq, sent, given, starts, words, passed):  # noqa: F811
    c, x = kvq.PagedCache("int8p", "int8p", 2, 4, device="cpu"), torch.zeros((70, 4, 128))
    B = 2 if starts else 70
    kw = dict(run_starts=i32(B + 1)) if starts else {}
    if given is not None:
        kw["max_run"] = given
    kvq.attn_tree(c, x, i32(B), i32(B, 2), i32(70, words), x.clone(), torch.zeros(64, dtype=torch.uint8), **kw)
    assert sent[0][1][8] == passed


def test_strided_rows_are_taken_as_they_are(kvq, sent):  # noqa: F811
    fused = torch.zeros((6, 8, 128))
    kvq.rope_runs(fused[:, :4], fused[:, 4:6], i32(6), torch.zeros(4, 128))
    a = sent[0][1]
    assert a[1] == a[4] == a[14] == a[16] == 1024 and a[0] == a[13] and a[3] == a[15] == a[0] + 4 * 4 * 128
    probs = torch.zeros((6, 12))
    kvq.verify_runs(probs[:, 1:10], i32(6), i32(6), None, i32(6), i32(6), i32(6))
    assert sent[1][1][1] == 12 and sent[1][1][5] == 9


def test_descriptors_of_all_layers_are_those_of_their_planes(kvq, sent):  # noqa: F811
    layers = [kvq.PagedCache("e4m3p", "e4m3p", 2, 4, layer=i, device="cpu") for i in range(3)]
    for _ in range(2):
        kvq.keep_runs(layers, i32(2), i32(2, 2), i32(6), i32(2), run_starts=i32(3))
        descs, n = sent[-1][1][:2]
        assert n == 3 and descs == b"".join(bytes(c.desc()) for c in layers)
        layers[1].v, layers[2].k_scale = torch.zeros_like(layers[1].v), torch.ones_like(layers[2].k_scale)
        layers[0].k.data = torch.zeros_like(layers[0].k)


def test_rotation_of_nothing_is_refused(kvq, sent):  # noqa: F811
    with pytest.raises(AssertionError):
        kvq.rope_runs(None, None, i32(2), torch.zeros(4, 128))
