"""kvq_map_runs, kvq_append_runs and kvq_attn_runs against the float64 oracle (GPU).

Maps and codes are functions of the inputs alone and must be equal; attention is held to the bound of its roundings
(tests/runs_cases.py), element by element.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from oracle import runs as R  # noqa: E402
from tests.runs_cases import (FMTS, attn_tolerance, lse_tolerance, pack, pages_of, random_codes, starts_of, tables,  # noqa: E402
                              unpack)


@pytest.fixture(scope="module")
def kvq():
    import quantized_kv_cache_kvq_gb300 as m

    m.load()
    return m


def dev(x, dtype=torch.int32):
    return torch.as_tensor(np.ascontiguousarray(x)).to("cuda", dtype)


def err_word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------------------------------------ maps
def run_map(kvq, new, lens, stack, count, table, max_rows, in_place=False):
    d = dict(new=dev(new), lens=dev(lens), stack=dev(stack), count=dev([count]), table=dev(table))
    B = len(new)
    d["starts"] = torch.full((B + 1,), -7, dtype=torch.int32, device="cuda")
    d["lens_out"] = d["lens"] if in_place else torch.full((B,), -7, dtype=torch.int32, device="cuda")
    d["count_out"] = d["count"] if in_place else torch.full((1,), -7, dtype=torch.int32, device="cuda")
    d["slots"] = torch.full((max_rows,), -7, dtype=torch.int32, device="cuda")
    d["pos"] = torch.full((max_rows,), -7, dtype=torch.int32, device="cuda")
    err = err_word()
    kvq.map_runs(d["new"], d["lens"], d["stack"], d["count"], d["table"], d["starts"], d["lens_out"], d["count_out"],
                 slot_mapping=d["slots"], positions=d["pos"], err=err)
    torch.cuda.synchronize()
    return {k: v.cpu().numpy() for k, v in d.items()}, int(err.item())


def check_map(got, ref):
    for a, b in (("starts", "run_starts"), ("lens_out", "seq_lens"), ("stack", "stack"), ("table", "table"), ("slots", "slots"),
                 ("pos", "positions")):
        assert np.array_equal(got[a], ref[b]), a
    assert got["count_out"][0] == ref["count"]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("batch,hi,new_hi,gone,fresh", [(1, 0, 1, 0, 0), (1, 40, 33, 0, 0), (7, 50, 20, .3, .3), (64, 700, 1, 0, 0),
                                                        (333, 90, 40, .4, .2), (1024, 60, 30, .2, .3), (1024, 200, 1, .9, 0)])
def test_map_equals_the_oracle(kvq, batch, hi, new_hi, gone, fresh, in_place):
    rng = np.random.default_rng(batch + hi)
    lens = np.where(rng.random(batch) < fresh, 0, rng.integers(0, hi + 1, batch))
    new = np.where(rng.random(batch) < gone, -1, rng.integers(0, new_hi + 1, batch))
    width = int(pages_of((lens + np.maximum(new, 0)).max())) + 1
    table, total = tables(rng, lens, width=width)
    spare = int(sum(max(0, pages_of(l + n) - pages_of(l)) for l, n in zip(lens, new) if n > 0)) + 2
    used = set(table[table >= 0].tolist())
    free = [p for p in range(total + spare) if p not in used]
    stack = np.full(total + spare, -9)
    stack[:len(free)] = rng.permutation(free)
    rows = int(np.maximum(new, 0).sum()) + 5
    ref = R.map_runs(new, lens, stack, len(free), table, rows)
    assert ref["ok"]
    got, err = run_map(kvq, new, lens, stack, len(free), table, rows, in_place)
    assert err == 0
    check_map(got, ref)


@pytest.mark.parametrize("kind,status", [("pages", 9), ("pages and rows", 5), ("rows", 5), ("width", 5), ("length", 5), ("count", 5), ("negative", 5),
                                         ("overflow", 5)])
def test_map_all_or_nothing(kvq, kind, status):
    new, lens, table = [20, -1, 3], [5, 17, 0], np.array([[4, -1, -1], [5, 6, -1], [-1, -1, -1]], dtype=np.int32)
    stack, count, rows = [1, 2, 3, 9, 9, 9], 3, 40
    if kind == "pages":
        new, count, rows = [40, 3, 40], 1, 83
    elif kind == "pages and rows":
        new, count = [40, 3, 40], 1
    elif kind == "rows":
        rows = 22
    elif kind == "width":
        new = [44, -1, 3]
    elif kind == "length":
        lens = [5, 49, 0]
    elif kind == "count":
        count = 7
    elif kind == "negative":
        lens = [5, -1, 0]
    elif kind == "overflow":
        stack, new = [1, 2, 3], [0, -1, 0]
    ref = R.map_runs(new, lens, stack, count, table, rows)
    assert not ref["ok"]
    got, err = run_map(kvq, new, lens, stack, count, table, rows)
    assert err == status
    check_map(got, ref)


def test_map_of_no_request_and_without_row_outputs(kvq):
    got, err = run_map(kvq, [], [], [3, 4], 2, np.zeros((0, 1)), 3)
    assert err == 0 and got["starts"].tolist() == [0] and got["count_out"].tolist() == [2] and got["slots"].tolist() == [-1] * 3
    t = [dev(x) for x in ([5], [0], [3, 4], [2], [[-1]])]
    starts, count = dev([0, 0]), dev([0])
    kvq.map_runs(*t, starts, t[1], count)
    assert starts.tolist() == [0, 5] and t[1].tolist() == [5] and count.tolist() == [1] and t[4].tolist() == [[4]]


# ------------------------------------------------------------------------------------------------ append
def make_cache(kvq, fmt, heads, pages, codes_k, codes_v, ek, ev):
    f16 = lambda e: torch.as_tensor(np.ascontiguousarray(2.0 ** e.T)).to("cuda", torch.float16).contiguous()  # noqa: E731
    return kvq.PagedCache.over(fmt, fmt, heads, pages, k=dev(pack(codes_k, fmt, "k"), torch.uint8),
                               v=dev(pack(codes_v, fmt, "v"), torch.uint8), k_scale=f16(ek), v_scale=f16(ev))


def check_cache(cache, fmt, heads, codes_k, codes_v, ek, ev):
    for plane, sc, codes, e in (("k", cache.k_scale, codes_k, ek), ("v", cache.v_scale, codes_v, ev)):
        assert np.array_equal(sc.cpu().double().numpy(), 2.0 ** e.T), plane
        assert np.array_equal(unpack(getattr(cache, plane).cpu().numpy(), heads, fmt, plane), codes), plane


APPENDS = [([1], [0], 1), ([1], [15], 2), ([1] * 9, [0, 1, 7, 14, 15, 16, 17, 31, 100], 3), ([16], [0], 8), ([37, 0, 5, 1], [3, 9, 0, 31], 4),
           ([300, 2], [11, 5], 2), ([17] * 70, list(range(70)), 1)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("new,old,heads", APPENDS)
def test_append_equals_the_oracle(kvq, fmt, dtype, new, old, heads):
    rng = np.random.default_rng(sum(new) + heads)
    lens = np.array(old) + new
    table, pages = tables(rng, lens)
    ck, cv = random_codes(rng, pages, heads, fmt), random_codes(rng, pages, heads, fmt)
    ek, ev = rng.integers(-9, -2, (pages, heads)), rng.integers(-9, -2, (pages, heads))
    cache = make_cache(kvq, fmt, heads, pages, ck, cv, ek, ev)
    n = int(sum(new))
    # rows of widely different size, so that scales grow by many steps and not at all
    fused = rng.standard_normal((n, 2 * heads, 128)) * 2.0 ** rng.integers(-6, 5, (n, 2 * heads, 1))
    t = torch.as_tensor(fused).to("cuda", torch.bfloat16 if dtype == "bf16" else torch.float32)
    x = t.double().cpu().numpy()
    k, v = t[:, :heads], t[:, heads:]  # slices of a fused projection
    starts = starts_of(new)
    R.append_runs(ck, ek, x[:, :heads], starts, lens, table, fmt)
    R.append_runs(cv, ev, x[:, heads:], starts, lens, table, fmt)
    err = err_word()
    kvq.append_runs(cache, k, v, dev(lens), dev(table), run_starts=None if new == [1] * len(new) else dev(starts), err=err)
    assert err.item() == 0
    check_cache(cache, fmt, heads, ck, cv, ek, ev)


@pytest.mark.parametrize("fmt", FMTS)
def test_append_token_by_token_and_a_reused_page(kvq, fmt):
    """A page filled one token at a time whose scale grows all along; then the page is reused: nothing of it is left."""
    rng = np.random.default_rng(2)
    ck, cv = random_codes(rng, 2, 2, fmt), random_codes(rng, 2, 2, fmt)
    ek, ev = np.full((2, 2), 9), np.full((2, 2), 9)
    cache = make_cache(kvq, fmt, 2, 2, ck, cv, ek, ev)
    table = np.array([[1]], dtype=np.int32)
    err = err_word()
    for lap in range(2):
        for t in range(16 if lap == 0 else 3):
            x = (rng.standard_normal((1, 4, 128)) * 1.9 ** (t - 4 * lap)).astype(np.float32)
            R.append_runs(ck, ek, x[:, :2], [0, 1], [t + 1], table, fmt)
            R.append_runs(cv, ev, x[:, 2:], [0, 1], [t + 1], table, fmt)
            d = torch.from_numpy(x).cuda()
            kvq.append_runs(cache, d[:, :2], d[:, 2:], dev([t + 1]), dev(table), err=err)
            check_cache(cache, fmt, 2, ck, cv, ek, ev)
    assert err.item() == 0


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("back", [16, 17, 20, 32])
def test_append_after_tokens_were_given_up(kvq, fmt, back):
    """A draft of large values is rejected down to ``back`` tokens: inside a page its scale stays, at a page's start it does not."""
    rng = np.random.default_rng(back)
    ck, cv = random_codes(rng, 4, 2, fmt), random_codes(rng, 4, 2, fmt)
    ek, ev = np.full((4, 2), -5), np.full((4, 2), -5)
    cache = make_cache(kvq, fmt, 2, 4, ck, cv, ek, ev)
    table = np.array([[2, 0, 3]], dtype=np.int32)
    err = err_word()
    for n, end, size in ((14, 14, 1.0), (21, 35, 40.0), (3, back + 3, 0.5), (1, back + 4, 0.01)):
        x = (rng.standard_normal((n, 4, 128)) * size).astype(np.float32)
        R.append_runs(ck, ek, x[:, :2], [0, n], [end], table, fmt)
        R.append_runs(cv, ev, x[:, 2:], [0, n], [end], table, fmt)
        d = torch.from_numpy(x).cuda()
        kvq.append_runs(cache, d[:, :2], d[:, 2:], dev([end]), dev(table), run_starts=dev([0, n]), err=err)
        check_cache(cache, fmt, 2, ck, cv, ek, ev)
    assert err.item() == 0


def test_a_cache_follows_its_planes(kvq):
    """Planes put into a cache after it was made are the ones that the calls use."""
    cache = kvq.PagedCache("int8p", "int8p", 1, 1)
    old = cache.k, cache.v, cache.k_scale, cache.v_scale
    cache.k, cache.v, cache.k_scale, cache.v_scale = (t.clone() for t in old)
    x = torch.ones((1, 1, 128), device="cuda")
    kvq.append_runs(cache, x, x, dev([1]), dev([[0]]))
    assert all(t.count_nonzero() == 0 for t in old)
    assert cache.k_scale.item() == cache.v_scale.item() == 2.0 ** -6  # 127 2^-7 < 1


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("kind,status", [("zeros", 0), ("tiny", 0), ("nan", 6), ("inf", 6), ("huge", 7), ("top", 0), ("bf16max", 7)])
def test_append_special_values(kvq, fmt, kind, status):
    rng = np.random.default_rng(4)
    x = rng.standard_normal((20, 2, 128)).astype(np.float32)
    if kind == "zeros":
        x[:] = 0
    elif kind == "tiny":
        x *= 1e-9
    elif kind == "nan":
        x[3, 0, 5] = np.nan
    elif kind == "inf":
        x[3, 0, 5], x[18, 0, 77] = np.inf, -np.inf
    elif kind == "huge":
        x[7, 0, 9] = R.QMAX[fmt] * 2.0 ** 15 * 3
    elif kind == "top":
        x[7, 0, 9] = R.QMAX[fmt] * 2.0 ** 15
    elif kind == "bf16max":
        x[7, 0, 9] = -3.3e38
    table = np.array([[2, 0]], dtype=np.int32)
    ck, cv = random_codes(rng, 3, 1, fmt), random_codes(rng, 3, 1, fmt)
    ek, ev = np.full((3, 1), -24), np.full((3, 1), 3)
    cache = make_cache(kvq, fmt, 1, 3, ck, cv, ek, ev)
    R.append_runs(ck, ek, x[:, :1], [0, 20], [20], table, fmt)
    R.append_runs(cv, ev, x[:, 1:], [0, 20], [20], table, fmt)
    err = err_word()
    d = torch.from_numpy(x).cuda()
    kvq.append_runs(cache, d[:, :1], d[:, 1:], dev([20]), dev(table), run_starts=dev([0, 20]), err=err)
    assert err.item() == status
    check_cache(cache, fmt, 1, ck, cv, ek, ev)


def test_append_skips_what_cannot_be(kvq):
    """A page outside the cache, a run longer than its context, a run outside the rows: reported, the others appended."""
    fmt, rng = "int8p", np.random.default_rng(6)
    for table, lens, starts in (([[7], [1]], [3, 3], [0, 3, 6]), ([[-1], [1]], [3, 3], [0, 3, 6]), ([[0], [1]], [2, 3], [0, 3, 6]),
                                ([[0], [1]], [17, 3], [0, 3, 6]), ([[0], [1]], [3, 3], [4, 3, 6]), ([[0], [1]], [3, 3], [-1, 3, 6])):
        table = np.array(table, dtype=np.int32)
        ck, cv = random_codes(rng, 2, 1, fmt), random_codes(rng, 2, 1, fmt)
        ek, ev = np.full((2, 1), -5), np.full((2, 1), -5)
        cache = make_cache(kvq, fmt, 1, 2, ck, cv, ek, ev)
        x = torch.randn(6, 2, 128, device="cuda")
        y = x.double().cpu().numpy()
        R.append_runs(ck, ek, y[3:, :1], [0, 3], [3], table[1:], fmt)
        R.append_runs(cv, ev, y[3:, 1:], [0, 3], [3], table[1:], fmt)
        err = err_word()
        kvq.append_runs(cache, x[:, :1], x[:, 1:], dev(lens), dev(table), run_starts=dev(starts), err=err)
        assert err.item() == 5
        check_cache(cache, fmt, 1, ck, cv, ek, ev)


# ------------------------------------------------------------------------------------------------ attention
def attention_case(kvq, fmt, dtype, lens, new, heads, group, seed=0, exps=(-7, -4), sm_scale=None, q_scale=1.0, behind=0, max_run=None,
                   spoil=True, bad_query=None):
    """Runs the call and checks every element; returns what it ran with.  bad_query: a (row, head) whose query holds a NaN; its
    output is NaN and every other row is as near to the formula as without it (not the same bits: the rows of a unit move
    their running maxima together)."""
    rng = np.random.default_rng(seed)
    lens, new = np.array(lens), np.array(new)
    table, pages = tables(rng, lens)
    ck, cv = random_codes(rng, pages, heads, fmt), random_codes(rng, pages, heads, fmt)
    ek, ev = rng.integers(exps[0], exps[1] + 1, (pages, heads)), rng.integers(exps[0], exps[1] + 1, (pages, heads))
    if spoil:  # what lies behind a context may hold anything: the largest codes, NaN bytes
        for s, n in enumerate(lens):
            if n % 16:
                for c in (ck, cv):
                    c[table[s, n // 16], :, n % 16:] = 255
    cache = make_cache(kvq, fmt, heads, pages, ck, cv, ek, ev)
    starts = starts_of(new)
    rows, Hq = int(new.sum()), heads * group
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    qkv = torch.as_tensor(rng.standard_normal((rows + behind, Hq + 3, 128)) * q_scale).to("cuda", dt)
    q = qkv[:, 1:Hq + 1] if Hq * 128 % 8 == 0 else qkv[:, 1:Hq + 1].contiguous()
    clean = q[:rows].double().cpu().numpy()
    if bad_query:
        q[bad_query][5] = float("nan")
    out = torch.full((rows + behind, Hq, 128), 7.0, dtype=dt, device="cuda")
    lse = torch.full((rows + behind, Hq), 7.0, device="cuda")
    max_run = max_run or max(1, int(new.max()))
    ws = torch.full((kvq.attn_runs_workspace_size(len(lens), rows + behind, max_run, heads, Hq, dt),), 255, dtype=torch.uint8,
                    device="cuda")
    err = err_word()
    single = bool((new == 1).all()) and not behind
    kw = dict(run_starts=None if single else dev(starts), max_run=max_run, lse=lse, sm_scale=sm_scale, err=err)
    args = (cache, q, dev(lens), dev(table), out, ws)
    kvq.attn_runs(*args, **kw)
    torch.cuda.synchronize()
    assert err.item() == 0
    scale = 128 ** -0.5 if sm_scale is None else sm_scale
    want, want_lse, pv, xa, low = R.attend(ck, ek, cv, ev, clean, starts, lens, table, scale, fmt)
    got, got_lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    if bad_query:
        assert np.all(np.isnan(got[bad_query])) and np.isnan(got_lse[bad_query])
        got[bad_query], got_lse[bad_query] = want[bad_query], want_lse[bad_query]
    assert np.all(got[rows:] == 7) and np.all(got_lse[rows:] == 7)
    got, got_lse = got[:rows], got_lse[:rows]
    off = np.abs(got - want) - attn_tolerance(want, pv, xa, low, dtype == "bf16")
    assert np.all(off <= 0), (float(off.max()), np.unravel_index(off.argmax(), off.shape))
    empty = np.isneginf(want_lse)
    assert np.array_equal(np.isneginf(got_lse), empty)
    assert np.all(np.abs(got_lse[~empty] - want_lse[~empty]) <= lse_tolerance(want_lse, xa)[~empty])
    return args, kw


LENS = [1, 2, 15, 16, 17, 31, 33, 127, 128, 129, 255, 300, 0]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("heads,group", [(1, 1), (2, 3), (3, 4), (4, 7), (2, 8)])
def test_decode_lengths_and_groups(kvq, fmt, dtype, heads, group):
    attention_case(kvq, fmt, dtype, LENS, [1] * len(LENS), heads, group)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("heads,group,new", [(2, 4, [2, 3, 4, 0, 1]), (1, 8, [2, 2, 1, 0, 2]), (3, 1, [5, 16, 9, 1, 0]),
                                             (2, 5, [3, 1, 2, 3, 0])])
def test_drafts(kvq, fmt, dtype, heads, group, new):
    attention_case(kvq, fmt, dtype, [300, 17, 16, 5, 130], new, heads, group, behind=3)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,new,heads,group", [
    ([64], [64], 1, 4), ([17], [17], 2, 1), ([200, 1, 77], [200, 1, 50], 2, 4), ([300, 64, 500, 33], [33, 1, 129, 20], 2, 7),
    ([513], [257], 1, 8), ([400, 400], [3, 150], 3, 3), ([130], [129], 1, 2), ([5, 600], [5, 300], 1, 1)])
def test_prompts_and_chunks(kvq, fmt, dtype, lens, new, heads, group):
    attention_case(kvq, fmt, dtype, lens, new, heads, group, behind=2)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_runs_longer_than_their_context_start_before_it(kvq, fmt, dtype):
    """Rows at positions below zero see nothing: 0 and -inf."""
    attention_case(kvq, fmt, dtype, [3, 0, 20], [5, 2, 1], 2, 2)
    attention_case(kvq, fmt, dtype, [3, 0, 40], [50, 30, 40], 1, 4)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("new", [[1, 1], [40, 90]])
def test_scales_far_apart(kvq, fmt, new):
    """Page scales over the whole range that the value product meets: the weights take the exponents."""
    attention_case(kvq, fmt, "bf16", [230, 95], new, 2, 4, exps=(-20, 2), q_scale=0.01)


@pytest.mark.parametrize("new", [[1, 1, 1], [30, 100, 1]])
def test_sharp_flat_and_negative_scales(kvq, new):
    lens = [100, 257, 40]
    attention_case(kvq, "int8p", "bf16", lens, new, 2, 4, q_scale=12.0)           # logits of hundreds: one token takes all
    attention_case(kvq, "int8p", "bf16", lens, new, 2, 4, sm_scale=0.0)           # a plain mean
    attention_case(kvq, "e4m3p", "bf16", lens, new, 2, 4, sm_scale=-0.2)
    attention_case(kvq, "e4m3p", "bf16", lens, new, 2, 4, q_scale=1e-30)
    attention_case(kvq, "e4m3p", "bf16", lens, new, 2, 4, q_scale=1e30, sm_scale=1e-31)


@pytest.mark.parametrize("fmt,dtype", [("e4m3p", "bf16"), ("int8p", "f32")])
@pytest.mark.parametrize("lens,new,heads,group", [([20000, 300], [1, 1], 1, 1), ([9000, 40, 7000], [1, 1, 1], 2, 3),
                                                  ([12000], [2], 1, 5), ([300, 11000], [0, 1], 4, 8)])
def test_few_requests_of_long_contexts(kvq, fmt, dtype, lens, new, heads, group):
    """Rows of hundreds of pieces, beside rows of a few; then with a query that is not finite."""
    attention_case(kvq, fmt, dtype, lens, new, heads, group, seed=7, behind=1)
    attention_case(kvq, fmt, dtype, lens, new, heads, group, seed=7, behind=1, bad_query=(0, 0))


CHUNKS = [([20, 100, 129, 257, 384, 513, 641], [5, 20, 9, 17, 20, 32, 31], 2, 4), ([3000, 1000, 5000], [6, 17, 32], 8, 4),
          ([3000, 900, 2500, 700, 50, 1], [6, 200, 32, 70, 1, 1], 4, 4), ([700, 2000, 300], [17, 128, 129], 3, 1),
          ([600 + 9 * i for i in range(40)], [3 + i % 14 for i in range(40)], 8, 8)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("lens,new,heads,group", CHUNKS)
def test_chunks_of_at_most_128_rows_among_others(kvq, fmt, lens, new, heads, group):
    """Units that fill one half of a tile's rows at most: of one key tile, of a few, cut anywhere, beside full ones."""
    attention_case(kvq, fmt, "bf16", lens, new, heads, group, seed=len(lens))


@pytest.mark.parametrize("q_scale", [30.0, 1e-3])
def test_chunks_with_sharp_and_flat_weights(kvq, q_scale):
    attention_case(kvq, "int8p", "bf16", [2000, 40, 900], [12, 30, 20], 2, 4, seed=5, q_scale=q_scale, exps=(-12, -3))


@pytest.mark.parametrize("fmt", FMTS)
def test_several_tiles_and_units_for_every_block(kvq, fmt):
    attention_case(kvq, fmt, "bf16", [2100, 900, 40, 700], [700, 900, 1, 3], 4, 2, behind=5)


def test_long_context_in_random_pages(kvq):
    attention_case(kvq, "int8p", "bf16", [20011, 31, 7000], [1, 1, 1], 2, 7)
    attention_case(kvq, "e4m3p", "bf16", [9001, 31], [40, 31], 1, 8)


@pytest.mark.parametrize("new", [[1, 1], [3, 40]])
def test_a_query_that_is_not_finite_stays_in_its_row(kvq, new):
    (cache, q, lens, table, out, ws), kw = attention_case(kvq, "int8p", "bf16", [50, 60], new, 2, 4)
    ref = out.clone()
    q[1, 5, 3] = float("nan")
    kvq.attn_runs(cache, q, lens, table, out, ws, **kw)
    assert out[1, 5].isnan().all()
    keep = torch.ones(out.shape[:2], dtype=torch.bool, device="cuda")
    keep[1, 5] = False
    assert torch.equal(out[keep], ref[keep])


@pytest.mark.parametrize("new,bad", [([1, 1, 1], 1), ([20, 30, 5], 1)])
def test_a_page_outside_the_cache_is_reported_and_the_others_are_right(kvq, new, bad):
    (cache, q, lens, table, out, ws), kw = attention_case(kvq, "e4m3p", "bf16", [50, 60, 70], new, 2, 4)
    ref = out.clone()
    for page in (-1, cache.num_pages, 1 << 30):
        table[bad, 0] = page
        kw["err"].zero_()
        kvq.attn_runs(cache, q, lens, table, out, ws, **kw)
        assert kw["err"].item() == 5
        starts = starts_of(new)
        assert torch.equal(out[:starts[bad]], ref[:starts[bad]]) and torch.equal(out[starts[bad + 1]:], ref[starts[bad + 1]:])
        # the request itself: its other tokens
        codes = [unpack(p.cpu().numpy(), 2, "e4m3p", n) for p, n in ((cache.k, "k"), (cache.v, "v"))]
        pages = table[bad, 1:4].cpu().numpy()
        k, v = ((R.values(c[pages], "e4m3p") * sc.cpu().double().numpy().T[pages][:, :, None, None]).transpose(1, 0, 2, 3).reshape(2, -1, 128)
                for c, sc in zip(codes, (cache.k_scale, cache.v_scale)))
        row, pos = starts[bad + 1] - 1, 60 - 16  # its last query sees tokens 16 .. 59
        for h in range(8):
            x = k[h // 4, :pos] @ q[row, h].double().cpu().numpy() / 128 ** 0.5
            w = np.exp(x - x.max())
            want = w @ v[h // 4, :pos] / w.sum()
            assert np.linalg.norm(out[row, h].double().cpu().numpy() - want) <= 0.01 * np.linalg.norm(want)


def test_runs_that_cannot_be_are_skipped(kvq):
    """A run past max_run, past the rows, backwards or with a length past its table: reported, its rows left as they were."""
    for starts, lens, max_run, wrong in (([0, 3, 6], [50, 60], 2, [0, 1]), ([0, 3, 9], [50, 60], 9, [1]), ([2, 1, 4], [50, 60], 4, [0]),
                                         ([0, 3, 6], [50, 65], 3, [1]), ([0, 3, 6], [-1, 60], 3, [0])):
        rng = np.random.default_rng(1)
        table, pages = tables(rng, [50, 60])
        c = random_codes(rng, pages, 1, "int8p")
        e = np.full((pages, 1), -5)
        cache = make_cache(kvq, "int8p", 1, pages, c, c, e, e)
        q = torch.randn(6, 4, 128, device="cuda").bfloat16()
        out = torch.full_like(q, 7.0)
        ws = torch.empty(kvq.attn_runs_workspace_size(2, 6, max_run, 1, 4, q.dtype), dtype=torch.uint8, device="cuda")
        err = err_word()
        kvq.attn_runs(cache, q, dev(lens), dev(table), out, ws, run_starts=dev(starts), max_run=max_run, err=err)
        assert err.item() == 5
        for s in range(2):
            if s not in wrong:
                a, b = starts[s], starts[s + 1]
                want, _, pv, xa, low = R.attend(c, e, c, e, q.double().cpu().numpy()[a:b], [0, b - a], lens[s:s + 1], table[s:s + 1], 128 ** -0.5, "int8p")
                assert np.all(np.abs(out[a:b].double().cpu().numpy() - want) <= attn_tolerance(want, pv, xa, low, True))


def test_runs_that_overlap_do_no_harm(kvq):
    """Run starts that go back and forth make more rows than there are: reported, nothing out of bounds."""
    B, rows = 64, 40
    starts = np.array([0, rows] * (B // 2) + [0], dtype=np.int32)
    rng = np.random.default_rng(1)
    table, pages = tables(rng, [64] * B)
    c = random_codes(rng, pages, 1, "int8p")
    e = np.full((pages, 1), -5)
    cache = make_cache(kvq, "int8p", 1, pages, c, c, e, e)
    for dt in (torch.float32, torch.bfloat16):
        q = torch.randn(rows, 4, 128, device="cuda", dtype=dt)
        ws = torch.empty(kvq.attn_runs_workspace_size(B, rows, rows, 1, 4, dt), dtype=torch.uint8, device="cuda")
        err = err_word()
        kvq.attn_runs(cache, q, dev([64] * B), dev(table), torch.empty_like(q), ws, run_starts=dev(starts), max_run=rows, err=err)
        assert err.item() == 5
        kvq.append_runs(cache, q[:, :1], q[:, 1:2], dev([64] * B), dev(table), run_starts=dev(starts), err=err)
        torch.cuda.synchronize()


def test_workspace_too_small_is_refused(kvq):
    (cache, q, lens, table, out, ws), kw = attention_case(kvq, "int8p", "bf16", [50], [1], 1, 2)
    with pytest.raises(kvq.KvqError) as e:
        kvq.attn_runs(cache, q, lens, table, out, ws[:-1], **kw)
    assert e.value.status == 3


# ------------------------------------------------------------------------------------------------ together
@pytest.mark.parametrize("fmt", FMTS)
def test_a_serving_loop_captured_once_and_replayed(kvq, fmt):
    """map -> append -> attention as one captured step on a side stream, replayed over a schedule with prompts, decoding,
    finished and new requests; state lives in the buffers.  Every step against the oracle."""
    rng = np.random.default_rng(9)
    B, width, pages, H, G, max_rows = 4, 8, 20, 2, 4, 96
    Hq = H * G
    st = dict(new=dev(np.zeros(B)), lens=dev(np.zeros(B)), stack=dev(np.arange(pages)), count=dev([pages]),
              table=dev(np.full((B, width), -1)), starts=dev(np.zeros(B + 1)), slots=dev(np.zeros(max_rows)), pos=dev(np.zeros(max_rows)))
    cache = kvq.PagedCache(fmt, fmt, H, pages)
    qkv = torch.zeros(max_rows, Hq + 2 * H, 128, dtype=torch.bfloat16, device="cuda")
    out = torch.zeros(max_rows, Hq, 128, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(max_rows, Hq, device="cuda")
    ws = torch.empty(kvq.attn_runs_workspace_size(B, max_rows, max_rows, H, Hq, qkv.dtype), dtype=torch.uint8, device="cuda")
    err = err_word()

    def step():
        kvq.map_runs(st["new"], st["lens"], st["stack"], st["count"], st["table"], st["starts"], st["lens"], st["count"],
                     slot_mapping=st["slots"], positions=st["pos"], err=err)
        kvq.append_runs(cache, qkv[:, Hq:Hq + H], qkv[:, Hq + H:], st["lens"], st["table"], run_starts=st["starts"], err=err)
        kvq.attn_runs(cache, qkv[:, :Hq], st["lens"], st["table"], out, ws, run_starts=st["starts"], max_run=max_rows, lse=lse, err=err)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()  # no tokens: nothing changes
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    zero = 128 if fmt == "int8p" else 0
    ck, cv = np.full((pages, H, 16, 128), 0), np.full((pages, H, 16, 128), 0)
    ek, ev = np.full((pages, H), -24), np.full((pages, H), -24)
    assert zero in (0, 128)
    lens, table, stack, count = np.zeros(B, int), np.full((B, width), -1), np.arange(pages), pages
    for new in ([20, 0, 33, 5], [1, 40, 1, 1], [1, 1, -1, 1], [1, 1, 60, 1], [-1, 2, 1, 3], [50, 1, 1, 1], [1, 1, 1, -1], [1, 1, 1, 17]):
        x = torch.as_tensor(rng.standard_normal(qkv.shape)).to("cuda", torch.bfloat16)
        qkv.copy_(x)
        st["new"].copy_(dev(new))
        out.fill_(7.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert err.item() == 0
        m = R.map_runs(new, lens, stack, count, table, max_rows)
        assert m["ok"]
        lens, table, stack, count = m["seq_lens"], m["table"], m["stack"], m["count"]
        assert np.array_equal(st["table"].cpu().numpy(), table) and np.array_equal(st["slots"].cpu().numpy(), m["slots"])
        assert st["lens"].tolist() == lens.tolist() and st["count"].item() == count
        y = x.double().cpu().numpy()
        starts, rows = m["run_starts"], int(m["run_starts"][-1])
        R.append_runs(ck, ek, y[:, Hq:Hq + H], starts, lens, table, fmt)
        R.append_runs(cv, ev, y[:, Hq + H:], starts, lens, table, fmt)
        want, want_lse, pv, xa, low = R.attend(ck, ek, cv, ev, y[:rows, :Hq], starts, lens, table, 128 ** -0.5, fmt)
        got = out.double().cpu().numpy()
        assert np.all(got[rows:] == 7)
        assert np.all(np.abs(got[:rows] - want) <= attn_tolerance(want, pv, xa, low, True))
        eager = torch.full_like(out, 7.0)
        kvq.attn_runs(cache, qkv[:, :Hq], st["lens"], st["table"], eager, ws, run_starts=st["starts"], max_run=max_rows)
        assert torch.equal(eager, out)  # bit for bit


def test_the_slot_map_feeds_the_per_token_layouts(kvq):
    """kvq_append takes kvq_map_runs' slot map, unused rows included, and kvq_decode_attn its tables and lengths."""
    B, H, Hq = 3, 2, 4
    t = dict(new=dev([20, 5, 1]), lens=dev([0, 0, 0]), stack=dev(np.arange(12)[::-1].copy()), count=dev([12]), table=dev(np.full((B, 4), -1)))
    starts, slots = dev(np.zeros(B + 1)), dev(np.zeros(32))
    err = err_word()
    kvq.map_runs(t["new"], t["lens"], t["stack"], t["count"], t["table"], starts, t["lens"], t["count"], slot_mapping=slots, err=err)
    cache = kvq.PagedCache("bf16", "bf16", H, 12)
    k, v = torch.randn(32, H, 128, device="cuda").bfloat16(), torch.randn(32, H, 128, device="cuda").bfloat16()
    kvq.append(cache, k, v, slots, err)
    q = torch.randn(B, Hq, 128, device="cuda").bfloat16()
    out = torch.empty(B, Hq, 128, device="cuda")
    ws = torch.empty(kvq.decode_workspace_size(B, H, Hq), dtype=torch.uint8, device="cuda")
    kvq.decode_attn(cache, q, t["table"], t["lens"], out, ws, err=err)
    assert err.item() == 0
    for s in range(B):
        a, b = starts.tolist()[s:s + 2]
        for h in range(Hq):
            x = (k[a:b, h // 2].double() @ q[s, h].double()) / 128 ** 0.5
            want = torch.softmax(x, 0) @ v[a:b, h // 2].double()
            assert (out[s, h].double() - want).norm() <= 2e-3 * want.norm()


def test_two_streams_with_a_workspace_each(kvq):
    cases = [attention_case(kvq, "int8p", "bf16", [3000, 70], [1, 1], 4, 4, seed=1), attention_case(kvq, "e4m3p", "bf16", [900, 70], [100, 3], 2, 4, seed=2)]
    refs = [a[4].clone() for a, _ in cases]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(10):
        for (a, kw), s in zip(cases, streams):
            kvq.attn_runs(*a, **dict(kw, stream=s))
    torch.cuda.synchronize()
    for (a, _), ref in zip(cases, refs):
        assert torch.equal(a[4], ref)

# ------------------------------------------------------------------------------------------------ limits
def test_offsets_past_32_bits(kvq):
    """Pages whose tiles lie beyond 4 GB of their plane, written and read."""
    H, G, pages = 8, 2, (1 << 32) // (8 * 2048) + 40
    for fmt in FMTS:
        cache = kvq.PagedCache(fmt, fmt, H, pages)
        assert cache.k.numel() > 1 << 32
        n = 50
        real = pages - 1 - np.arange(4)
        table, local = dev([real]), np.array([[0, 1, 2, 3]], dtype=np.int32)
        x = torch.randn(n, 2 * H + H * G, 128, device="cuda").bfloat16()
        y = x.double().cpu().numpy()
        err = err_word()
        kvq.append_runs(cache, x[:, :H], x[:, H:2 * H], dev([n]), table, run_starts=dev([0, n]), err=err)
        ck, cv = np.zeros((4, H, 16, 128), np.int64), np.zeros((4, H, 16, 128), np.int64)
        ek, ev = np.zeros((4, H), np.int64), np.zeros((4, H), np.int64)
        R.append_runs(ck, ek, y[:, :H], [0, n], [n], local, fmt)
        R.append_runs(cv, ev, y[:, H:2 * H], [0, n], [n], local, fmt)
        tiles = cache.k.view(pages, H, 2048)[torch.as_tensor(real.copy())].cpu().numpy()
        assert np.array_equal(unpack(tiles.reshape(-1, 2048), H, fmt, "k"), ck)
        q = x[:, 2 * H:]
        for rows in (n, 1):  # as a prompt and as one token
            out = torch.empty(rows, H * G, 128, dtype=torch.bfloat16, device="cuda")
            ws = torch.empty(kvq.attn_runs_workspace_size(1, rows, rows, H, H * G, q.dtype), dtype=torch.uint8, device="cuda")
            kvq.attn_runs(cache, q[n - rows:], dev([n]), table, out, ws, run_starts=dev([0, rows]), max_run=rows, err=err)
            want, _, pv, xa, low = R.attend(ck, ek, cv, ev, y[n - rows:, 2 * H:], [0, rows], [n], local, 128 ** -0.5, fmt)
            assert np.all(np.abs(out.double().cpu().numpy() - want) <= attn_tolerance(want, pv, xa, low, True))
        assert err.item() == 0
        del cache, tiles


def test_a_context_past_the_limit_is_refused(kvq):
    wide = torch.zeros(1, (1 << 26) + 1, dtype=torch.int32, device="cuda")
    cache = kvq.PagedCache("int8p", "int8p", 1, 1)
    x = torch.randn(1, 4, 128, device="cuda").bfloat16()
    out = torch.full((1, 4, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(kvq.attn_runs_workspace_size(1, 1, 1, 1, 4, x.dtype), dtype=torch.uint8, device="cuda")
    err = err_word()
    kvq.attn_runs(cache, x, dev([(1 << 30) + 1]), wide, out, ws, err=err)
    assert err.item() == 5 and torch.all(out == 7)
    err.zero_()
    before = cache.k.clone()
    kvq.append_runs(cache, x[:, :1], x[:, 1:2], dev([(1 << 30) + 1]), wide, err=err)
    assert err.item() == 5 and torch.equal(cache.k, before)
    err.zero_()
    lens, count, starts = dev([1 << 30]), dev([2]), dev([9, 9])
    kvq.map_runs(dev([1]), lens, dev([0, 0]), count, wide, starts, lens, count, err=err)
    assert err.item() == 5 and lens.tolist() == [1 << 30] and starts.tolist() == [0, 0] and count.tolist() == [2]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_the_largest_batch(kvq, dtype):
    rng = np.random.default_rng(8)
    lens = rng.integers(0, 40, 1024)
    attention_case(kvq, "int8p", dtype, lens, [1] * 1024, 1, 2)
    new = np.minimum(lens, rng.integers(0, 4, 1024))
    new[[3, 700]] = np.minimum(lens[[3, 700]], 30)
    attention_case(kvq, "e4m3p", dtype, lens, new, 1, 2, max_run=30)


@pytest.mark.parametrize("new", [[1, 1], [2, 1], [90, 200]])
def test_the_same_call_gives_the_same_bits(kvq, new):
    (cache, q, lens, table, out, ws), kw = attention_case(kvq, "e4m3p", "bf16", [3000, 700], new, 4, 4)
    ref, ref_lse = out.clone(), kw["lse"].clone()
    for fill in (0, 255, 127):  # whatever the workspace holds
        ws.fill_(fill)
        out.fill_(0)
        kvq.attn_runs(cache, q, lens, table, out, ws, **kw)
        assert torch.equal(out, ref) and torch.equal(kw["lse"], ref_lse)


def test_a_cache_without_pages(kvq):
    """Nothing can be read: every entry is outside the cache."""
    cache = kvq.PagedCache.over("int8p", "int8p", 1, 0, k=torch.empty(0, 2048, dtype=torch.uint8, device="cuda"),
                                v=torch.empty(0, 2048, dtype=torch.uint8, device="cuda"),
                                k_scale=torch.empty(1, 0, dtype=torch.float16, device="cuda"),
                                v_scale=torch.empty(1, 0, dtype=torch.float16, device="cuda"))
    q = torch.randn(40, 4, 128, device="cuda").bfloat16()
    ws = torch.empty(kvq.attn_runs_workspace_size(1, 40, 40, 1, 4, q.dtype), dtype=torch.uint8, device="cuda")
    with pytest.raises(kvq.KvqError):  # planes of nothing have no address
        kvq.attn_runs(cache, q, dev([40]), dev([[0, 0, 0]]), torch.empty_like(q), ws, run_starts=dev([0, 40]), max_run=40)


def test_empty_calls(kvq):
    cache = kvq.PagedCache("int8p", "int8p", 2, 2)
    x = torch.empty(0, 2, 128, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(16, dtype=torch.uint8, device="cuda")
    kvq.append_runs(cache, x, x, dev([]), dev(np.zeros((0, 1))))
    kvq.attn_runs(cache, x, dev([]), dev(np.zeros((0, 1))), torch.empty_like(x), ws)
    torch.cuda.synchronize()
