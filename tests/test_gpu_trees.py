"""Trees of drafted tokens against the oracle (GPU): masks, rotation, attention, verification, the kept path.

Masks, paths, tokens, codes and scales are functions of the inputs alone and must be equal; rotation and attention are held to the bound
of their roundings, element by element.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from oracle import trees as T  # noqa: E402
from tests.runs_cases import FMTS, attn_tolerance, lse_tolerance, random_codes, starts_of, tables  # noqa: E402
from tests.test_gpu_runs import check_cache, dev, err_word, make_cache  # noqa: E402
from tests.tree_cases import distribution, random_trees  # noqa: E402


@pytest.fixture(scope="module")
def kvq():
    import quantized_kv_cache_kvq_gb300 as m

    m.load()
    return m


# ------------------------------------------------------------------------------------------------ masks
@pytest.mark.parametrize("ns,words", [([1], 1), ([7, 0, 1, 32], 1), ([33, 64, 65, 2], 3), ([200, 31], 7), ([1024, 5], 32), ([100], 40), ([1000] * 3, 32)])
@pytest.mark.parametrize("spread", [1, 3, 1024])
def test_masks_and_positions(kvq, ns, words, spread):
    rng = np.random.default_rng(sum(ns) + spread)
    parents, starts = random_trees(rng, ns, spread), starts_of(ns)
    lens = np.array(ns) + rng.integers(0, 50, len(ns))
    rows = int(starts[-1])
    want, pos = T.tree_runs(parents, starts, lens, words)
    mask, positions = torch.full((rows + 3, words), 7, dtype=torch.int32, device="cuda"), torch.full((rows + 3,), 7, dtype=torch.int32, device="cuda")
    err = err_word()
    full = np.concatenate([parents, [0, 0, 0]])
    kvq.tree_runs(dev(full), dev(lens), mask, positions=positions, run_starts=dev(starts), err=err)
    assert err.item() == 0
    assert np.array_equal(mask[:rows].cpu().numpy(), want) and np.array_equal(positions[:rows].cpu().numpy(), pos)
    assert torch.all(mask[rows:] == 7) and torch.all(positions[rows:] == 7)
    again = torch.zeros_like(mask)
    kvq.tree_runs(dev(full), dev(lens), again, run_starts=dev(starts))
    assert np.array_equal(again[:rows].cpu().numpy(), want)


def test_masks_of_single_tokens_and_full_batches(kvq):
    mask, positions = torch.zeros((1024, 2), dtype=torch.int32, device="cuda"), torch.zeros(1024, dtype=torch.int32, device="cuda")
    lens = torch.arange(1, 1025, dtype=torch.int32, device="cuda")
    kvq.tree_runs(dev([-1] * 1024), lens, mask, positions=positions)
    assert torch.all(mask[:, 0] == 1) and torch.all(mask[:, 1] == 0) and torch.equal(positions, lens - 1)


@pytest.mark.parametrize("kind", ["forward", "itself", "low", "long", "longer than its context", "starts"])
def test_masks_of_what_cannot_be(kvq, kind):
    """Reported; the other request's rows are right."""
    parents, starts, lens, words = [-1, 0, 1, 0, -1, 0, 1], [0, 4, 7], [9, 8], 1
    first_is_written = True
    if kind == "forward":
        parents[1] = 3
    elif kind == "itself":
        parents[1] = 1
    elif kind == "low":
        parents[1] = -2
    elif kind == "long":
        parents, starts, lens, first_is_written = [-1] + [0] * 39 + [-1, 0, 1], [0, 40, 43], [60, 8], False
    elif kind == "longer than its context":
        lens, first_is_written = [3, 8], False
    else:
        starts, first_is_written = [5, 4, 7], False
    mask, positions = torch.full((len(parents), words), 7, dtype=torch.int32, device="cuda"), torch.full((len(parents),), 77, dtype=torch.int32, device="cuda")
    err = err_word()
    kvq.tree_runs(dev(parents), dev(lens), mask, positions=positions, run_starts=dev(starts), err=err)
    assert err.item() == 5
    assert mask[-3:, 0].tolist() == [1, 3, 7] and positions[-3:].tolist() == [5, 6, 7]
    if first_is_written:  # a parent that cannot be is none
        assert mask[:4, 0].tolist() == [1, 2, 6, 9] and positions[:4].tolist() == [5, 5, 6, 6]
    else:
        assert torch.all(mask[:-3] == 7) and torch.all(positions[:-3] == 77)


# ------------------------------------------------------------------------------------------------ rotation
def cos_sin(n):
    theta = 1e6 ** (-np.arange(64) / 64)
    a = np.arange(n)[:, None] * theta
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def rope_tolerance(x, weight, eps, positions, cs, bf16):
    """Norm: the sum of 128 squares in binary32 (each term rounded once, at most 128 additions: 2^-17 relative, halved by the root), its
    reciprocal root (2^-22), two products (2^-23): less than 2^-17 of every normed value.  Rotation: a product, a fused one and its
    sum, 2^-23 of |a c| + |b s| together.  bf16: half a step of the result, 2^-8."""
    size = T.rope(np.abs(x), None if weight is None else np.abs(weight), eps, positions, np.abs(cs) * np.where(np.arange(128) < 64, 1, -1))
    size = np.concatenate([size[..., :64], np.abs(T.rope(np.abs(x), None if weight is None else np.abs(weight), eps, positions, np.abs(cs)))[..., 64:]], -1)
    return (2.0 ** -17 if weight is not None else 0) * size + 2.0 ** -23 * size, 2.0 ** -8 if bf16 else 2.0 ** -24


def check_rope(got, x, weight, eps, positions, cs, bf16):
    want = T.rope(x, weight, eps, positions, cs)
    abs_tol, rel = rope_tolerance(x, weight, eps, positions, cs, bf16)
    off = np.abs(got - want) - (abs_tol * (1 + rel) + rel * np.abs(want) + 1e-37)
    assert np.all(off <= 0), float(off.max())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("norm", [(True, True), (True, False), (False, False)])
@pytest.mark.parametrize("rows,hq,hk", [(1, 1, 1), (7, 5, 3), (64, 32, 8), (33, 28, 4), (2, 64, 9)])
def test_rope(kvq, dtype, norm, rows, hq, hk):
    rng = np.random.default_rng(rows + hq)
    cs, behind = cos_sin(200), 2
    fused = torch.as_tensor(rng.standard_normal((rows + behind, hq + 2 * hk, 128)) * 2.0 ** rng.integers(-9, 9, (rows + behind, hq + 2 * hk, 1))).to("cuda", dtype)
    q, k = fused[:, :hq], fused[:, hq:hq + hk]
    was = fused.clone()
    positions = rng.integers(0, 200, rows + behind)
    w = [torch.as_tensor(rng.standard_normal(128)).to("cuda", torch.float32) if n else None for n in norm]
    x = [t.double().cpu().numpy()[:rows] for t in (q, k)]
    wn = [None if t is None else t.double().cpu().numpy() for t in w]
    starts = dev([0, rows // 2, rows])
    err = err_word()
    kw = dict(q_weight=w[0], k_weight=w[1], eps=1e-5, run_starts=starts, err=err)
    outs = torch.full_like(q.contiguous(), 7), torch.full((rows + behind, hk + 1, 128), 7, dtype=dtype, device="cuda")[:, 1:]
    kvq.rope_runs(q, k, dev(positions), dev(cs, torch.float32), q_out=outs[0], k_out=outs[1], **kw)
    assert err.item() == 0 and torch.equal(fused, was)
    for got, xi, wi in zip(outs, x, wn):
        assert torch.all(got[rows:] == 7)
        check_rope(got[:rows].double().cpu().numpy(), xi, wi, 1e-5, positions[:rows], cs, dtype is torch.bfloat16)
    kvq.rope_runs(q, k, dev(positions), dev(cs, torch.float32), **kw)  # in place, the values' heads untouched
    assert torch.equal(q[:rows], outs[0][:rows]) and torch.equal(k[:rows], outs[1][:rows])
    assert torch.equal(fused[:, hq + hk:], was[:, hq + hk:]) and torch.equal(fused[rows:], was[rows:])
    if not norm[0]:
        alone = torch.zeros_like(outs[0])
        kvq.rope_runs(was[:, :hq], None, dev(positions), dev(cs, torch.float32), q_out=alone, err=err)
        assert torch.equal(alone[:rows], outs[0][:rows]) and err.item() == 0
        kvq.rope_runs(None, was[:, hq:hq + hk], dev(positions), dev(cs, torch.float32), run_starts=starts, err=err)
        assert torch.equal(was[:rows, hq:hq + hk], outs[1][:rows]) and err.item() == 0


@pytest.mark.parametrize("size", [1e-25, 1e-38, 1e18, 1e30, 2e38])
def test_rope_norms_of_extreme_rows(kvq, size):
    """Squares that leave binary32."""
    rng = np.random.default_rng(3)
    x = rng.uniform(0.5, 1, (2, 3, 128)) * size
    t = torch.as_tensor(x).to("cuda", torch.float32)
    w = torch.ones(128, device="cuda")
    cs = cos_sin(5)
    out = torch.zeros_like(t)
    kvq.rope_runs(t, None, dev([0, 4]), dev(cs, torch.float32), q_weight=w, eps=0.0, q_out=out)
    check_rope(out.double().cpu().numpy(), t.double().cpu().numpy(), np.ones(128), 0.0, np.array([0, 4]), cs, False)


def test_rope_of_zeros_and_of_what_is_not_finite(kvq):
    t = torch.zeros((3, 1, 128), device="cuda")
    t[1, 0, 5], t[2, 0, 70] = float("nan"), float("inf")
    out = torch.full_like(t, 7)
    kvq.rope_runs(t, None, dev([1, 1, 1]), dev(cos_sin(2), torch.float32), q_weight=torch.ones(128, device="cuda"), q_out=out)
    assert torch.all(out[0] == 0) and torch.all(torch.isnan(out[1])) and torch.isnan(out[2, 0, 70])


@pytest.mark.parametrize("bad", [-1, 5, 1 << 30])
def test_rope_positions_outside_the_table(kvq, bad):
    t = torch.randn((3, 40, 128), device="cuda")
    out, want, err = torch.full_like(t, 7), torch.zeros_like(t), err_word()
    kvq.rope_runs(t, None, dev([1, bad, 2]), dev(cos_sin(5), torch.float32), q_out=out, err=err)
    assert err.item() == 5 and torch.all(out[1] == 7)
    kvq.rope_runs(t, None, dev([1, 0, 2]), dev(cos_sin(5), torch.float32), q_out=want)
    assert torch.equal(out[0], want[0]) and torch.equal(out[2], want[2])
    for end in (-1, 4):
        err.zero_()
        out.fill_(7)
        kvq.rope_runs(t, None, dev([1, 0, 2]), dev(cos_sin(5), torch.float32), q_out=out, run_starts=dev([0, end]), err=err)
        assert err.item() == 5 and torch.all(out == 7)


# ------------------------------------------------------------------------------------------------ attention
def tree_case(kvq, fmt, dtype, lens, new, heads, group, seed=0, spread=3, behind=0, max_run=None, masks="tree", exps=(-7, -4), sm_scale=None, q_scale=1.0):
    rng = np.random.default_rng(seed)
    lens, new = np.array(lens), np.array(new)
    table, pages = tables(rng, lens)
    ck, cv = random_codes(rng, pages, heads, fmt), random_codes(rng, pages, heads, fmt)
    ek, ev = rng.integers(exps[0], exps[1] + 1, (pages, heads)), rng.integers(exps[0], exps[1] + 1, (pages, heads))
    for s, n in enumerate(lens):  # what lies behind a context may hold anything: the largest codes, NaN bytes
        if n % 16:
            for c in (ck, cv):
                c[table[s, n // 16], :, n % 16:] = 255
    cache = make_cache(kvq, fmt, heads, pages, ck, cv, ek, ev)
    starts = starts_of(new)
    rows, Hq = int(new.sum()), heads * group
    words = (int(new.max()) + 31) // 32 + 1
    if masks == "tree":
        mask = T.tree_runs(random_trees(rng, new, spread), starts, lens, words)[0]
    elif masks == "none":
        mask = np.zeros((rows, words), np.int32)
    else:  # any bits, those behind the run among them
        mask = rng.integers(-2 ** 31, 2 ** 31, (rows, words)).astype(np.int32)
    mask = np.concatenate([mask, np.full((behind, words), -1, np.int32)])
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    qkv = torch.as_tensor(rng.standard_normal((rows + behind, Hq + 3, 128)) * q_scale).to("cuda", dt)
    q = qkv[:, 1:Hq + 1]
    out = torch.full((rows + behind, Hq, 128), 7.0, dtype=dt, device="cuda")
    lse = torch.full((rows + behind, Hq), 7.0, device="cuda")
    max_run = max_run or int(new.max())
    ws = torch.full((kvq.attn_tree_workspace_size(len(lens), rows + behind, max_run, heads, Hq, dt),), 255, dtype=torch.uint8, device="cuda")
    err = err_word()
    args = (cache, q, dev(lens), dev(table), dev(mask), out, ws)
    kw = dict(run_starts=None if bool((new == 1).all()) and not behind else dev(starts), max_run=max_run, lse=lse, sm_scale=sm_scale, err=err)
    kvq.attn_tree(*args, **kw)
    torch.cuda.synchronize()
    assert err.item() == 0
    scale = 128 ** -0.5 if sm_scale is None else sm_scale
    want, want_lse, pv, xa, low = T.attend_tree(ck, ek, cv, ev, q[:rows].double().cpu().numpy(), starts, lens, table, mask, scale, fmt)
    got, got_lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.all(got[rows:] == 7) and np.all(got_lse[rows:] == 7)
    got, got_lse = got[:rows], got_lse[:rows]
    off = np.abs(got - want) - attn_tolerance(want, pv, xa, low, dtype == "bf16")
    assert np.all(off <= 0), (float(off.max()), np.unravel_index(off.argmax(), off.shape))
    empty = np.isneginf(want_lse)
    assert np.array_equal(np.isneginf(got_lse), empty) and np.all(got[empty] == 0)
    assert np.all(np.abs(got_lse[~empty] - want_lse[~empty]) <= lse_tolerance(want_lse, xa)[~empty])
    return args, kw


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("heads,group", [(1, 1), (2, 4), (1, 7), (2, 8)])
@pytest.mark.parametrize("lens,new", [([1], [1]), ([5, 5], [5, 5]), ([300, 17, 16, 5, 130], [4, 3, 2, 0, 1]), ([33, 160, 31], [17, 9, 31]),
                                      ([140, 70], [64, 33])])
def test_trees_over_the_cache(kvq, fmt, dtype, heads, group, lens, new):
    tree_case(kvq, fmt, dtype, lens, new, heads, group, seed=len(lens), behind=2)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("masks", ["none", "any"])
def test_any_mask_and_rows_that_see_nothing(kvq, fmt, dtype, masks):
    tree_case(kvq, fmt, dtype, [8, 40, 41, 77, 3], [8, 40, 20, 33, 1], 2, 2, masks=masks, behind=1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("before", [0, 1, 15, 16, 17, 31, 100, 127, 128, 129])
def test_a_run_may_begin_anywhere(kvq, dtype, before):
    """The run's first page, key tile and mask word at every offset to each other."""
    tree_case(kvq, "int8p", dtype, [before + 37, before + 64, before + 3], [37, 64, 3], 1, 4, seed=before)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("new,lens,group", [([200], [260], 1), ([130, 1], [130, 900], 2), ([520], [530], 1), ([24, 7, 64], [2100, 1500, 700], 4)])
def test_large_trees_and_long_contexts(kvq, fmt, new, lens, group):
    tree_case(kvq, fmt, "bf16", lens, new, 1, group, seed=9)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scales_far_apart_and_large_logits(kvq, dtype):
    tree_case(kvq, "int8p", dtype, [90, 200], [21, 9], 2, 4, exps=(-16, -1), seed=5)
    tree_case(kvq, "e4m3p", dtype, [90, 200], [21, 9], 2, 4, q_scale=6.0, seed=6)
    tree_case(kvq, "int8p", dtype, [90, 200], [21, 9], 2, 4, sm_scale=-0.05, seed=7)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("new", [[3, 2], [25, 9], [64, 40]])
def test_a_chain_is_attn_runs(kvq, dtype, new):
    """The mask of a chain is causal: the same values to rounding; and a call repeats its bits."""
    args, kw = tree_case(kvq, "int8p", dtype, [400, 300], new, 2, 4, spread=1)
    out, lse = args[5].clone(), kw["lse"].clone()
    kvq.attn_tree(*args, **kw)
    assert torch.equal(out, args[5]) and torch.equal(lse, kw["lse"])
    cache, q, lens, table, _, o, _ = args
    ws = torch.empty(kvq.attn_runs_workspace_size(2, q.shape[0], kw["max_run"], 2, 8, q.dtype), dtype=torch.uint8, device="cuda")
    kvq.attn_runs(cache, q, lens, table, o, ws, **kw)
    torch.testing.assert_close(o.float(), out.float(), rtol=2e-2 if dtype == "bf16" else 1e-4, atol=2e-2 if dtype == "bf16" else 1e-4)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [5, 40])
def test_attention_of_what_cannot_be(kvq, dtype, n):
    """A run longer than max_run, a length beyond the table, a page outside the cache: reported; the other request is right."""
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    rng = np.random.default_rng(1)
    codes, exps = random_codes(rng, 8, 1, "int8p"), np.full((8, 1), -6)
    cache = make_cache(kvq, "int8p", 1, 8, codes, codes, exps, exps)
    q = torch.randn((n + 5, 2, 128), device="cuda").to(dt)
    mask = torch.full((n + 5, 2), -1, dtype=torch.int32, device="cuda")
    good = [[0, 1, 2, 3], [4, 5, 6, 7]]

    def call(lens, table, starts, max_run):
        out, err = torch.full_like(q, 7), err_word()
        ws = torch.empty(kvq.attn_tree_workspace_size(2, n + 5, max_run, 1, 2, dt), dtype=torch.uint8, device="cuda")
        kvq.attn_tree(cache, q, dev(lens), dev(table), mask, out, ws, run_starts=dev(starts), max_run=max_run, err=err)
        return out, err.item()

    want, status = call([60, 50], good, [0, n, n + 5], n)
    assert status == 0
    for lens, table, starts, max_run in (([60, 50], good, [0, n, n + 5], n - 1 if n > 6 else n), ([65, 50], good, [0, n, n + 5], n),
                                         ([-1, 50], good, [0, n, n + 5], n), ([60, 50], [[0, 1, 9, 3], good[1]], [0, n, n + 5], n),
                                         ([60, 50], good, [n + 1, n, n + 5], n)):
        out, status = call(lens, table, starts, max_run)
        assert status == 5 or max_run == n and lens == [60, 50] and table == good and starts[0] == 0
        torch.testing.assert_close(out[n:].float(), want[n:].float(), rtol=2e-2, atol=2e-2)


# ------------------------------------------------------------------------------------------------ verification
def verify_case(kvq, how, dtype, ns, V, seed, spread=3, stride=None, sharp=2.0):
    rng = np.random.default_rng(seed)
    rows, starts = sum(ns), starts_of(ns)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    parents = random_trees(rng, ns, spread)
    base = [distribution(rng, V, sharp) for _ in range(rows)]

    def held(x, like):
        x = torch.as_tensor(np.stack(x)).to("cuda", dt) if rows else torch.zeros((0, V), dtype=dt, device="cuda")
        if stride:
            x = torch.cat([torch.full((rows, stride[0]), 0.7, dtype=dt, device="cuda"), x, torch.full((rows, stride[1]), 0.9, dtype=dt, device="cuda")], 1)
            x = x[:, stride[0]:stride[0] + V]
        return x

    target = held([rng.standard_normal(V) * 4 for _ in range(rows)] if how == "greedy" else base, None)
    draft = held([(0.6 * p + 0.4 * distribution(rng, V, sharp)).astype(np.float32) for p in base], None) if how == "draft" else None
    tn = target.float().cpu().numpy()
    dn = None if draft is None else draft.float().cpu().numpy()
    # children that are likely to be accepted: drawn from the parent's distribution, some of them twice
    tokens = np.zeros(rows, dtype=np.int64)
    for s in range(len(ns)):
        for i in range(1, ns[s]):
            p = (dn if dn is not None else tn)[starts[s] + parents[starts[s] + i]].astype(np.float64)
            tokens[starts[s] + i] = rng.choice(V, p=p / p.sum()) if how == "draft" or rng.random() < 0.3 and how == "target" else np.argsort(-p)[min(V - 1, rng.integers(0, 3))]
    uniform = None if how == "greedy" else rng.random((rows, 2)).astype(np.float32)
    want = T.verify_runs(tn, dn, tokens, parents, uniform, starts)
    behind = 2
    keep = torch.full((rows,), 7, dtype=torch.int32, device="cuda")
    kept, following, err = dev([7] * len(ns)), dev([7] * len(ns)), err_word()
    lens = dev(np.array(ns) + behind)
    single = ns == [1] * len(ns)
    args = (target, dev(tokens), dev(parents), None if uniform is None else dev(uniform, torch.float32), keep, kept, following)
    kw = dict(draft=draft, seq_lens=lens, seq_lens_out=lens, run_starts=None if single else dev(starts), err=err)
    kvq.verify_runs(*args, **kw)
    assert err.item() == 0
    assert kept.tolist() == want[1].tolist() and following.tolist() == want[2].tolist()
    assert keep.tolist() == want[0].tolist() and lens.tolist() == (want[1] + behind).tolist()
    return want, args, kw


@pytest.mark.parametrize("how", ["greedy", "target", "draft"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("ns,V", [([1], 1), ([1, 1], 3), ([4, 0, 9], 17), ([12, 30, 1, 0, 7], 1000), ([20, 5], 4099), ([6, 7], 32000)])
def test_verification(kvq, how, dtype, ns, V):
    for seed in range(4):
        verify_case(kvq, how, dtype, ns, V, seed)


@pytest.mark.parametrize("how", ["target", "draft"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_verification_of_flat_distributions(kvq, how, dtype):
    """Where many tokens are about as likely, a sum that is a little off finds another token."""
    for seed in range(3):
        verify_case(kvq, how, dtype, [3, 8], 20011, seed, spread=8, sharp=0.02)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("stride", [(0, 5), (1, 2), (3, 9), (8, 8), (7, 0)])
@pytest.mark.parametrize("how", ["greedy", "target", "draft"])
def test_verification_of_rows_at_any_alignment(kvq, how, dtype, stride):
    verify_case(kvq, how, dtype, [5, 6], 517, 1, stride=stride)


def test_verification_of_long_chains_wide_trees_and_a_full_batch(kvq):
    verify_case(kvq, "draft", "f32", [1024], 33, 0, spread=1, sharp=0.3)
    verify_case(kvq, "draft", "f32", [700], 40, 0, spread=1024)
    verify_case(kvq, "target", "f32", [1024, 1024], 5, 1, spread=4)
    verify_case(kvq, "greedy", "bf16", [1] * 1024, 50, 2)
    verify_case(kvq, "draft", "f32", [2] * 1024, 50, 2)


def test_largest_vocabulary_and_one_hot_rows(kvq):
    V = 1 << 19
    t = torch.zeros((3, V), device="cuda")
    t[0, V - 1], t[1, 0], t[2, 77] = 1.0, 1.0, 1.0
    args = [dev([0, V - 1, 0]), dev([-1, 0, 1]), torch.tensor([[0, 0.999], [0.5, 0], [0.9, 0.5]], device="cuda")]
    for draft in (None, t):
        keep, kept, following, err = dev([7] * 3), dev([7]), dev([7]), err_word()
        kvq.verify_runs(t, *args, keep, kept, following, draft=draft, run_starts=dev([0, 3]), err=err)
        assert keep.tolist() == [0, 1, 2] and kept.item() == 3 and following.item() == 77 and err.item() == 0
    full = torch.ones((1, V), device="cuda")  # the largest sum there is
    keep, kept, following = dev([7]), dev([7]), dev([7])
    for u, tok in ((0.0, 0), (0.5, V // 2), (1 - 2.0 ** -24, V - 1)):
        kvq.verify_runs(full, dev([0]), dev([-1]), torch.tensor([[0.0, u]], device="cuda"), keep, kept, following)
        assert following.item() == tok
    kvq.verify_runs(full, dev([0]), dev([-1]), None, keep, kept, following)
    assert following.item() == 0  # equal scores: the lowest


def test_verification_where_the_residual_vanishes(kvq):
    """q = p in most places: a child whose p is 0 is refused, and what is left is 0 everywhere: the token is drawn from p."""
    p = torch.tensor([[0.5, 0.5, 0.0, 0.0]] * 2, device="cuda")
    q = torch.tensor([[0.5, 0.5, 0.5, 0.0]] * 2, device="cuda")
    u = torch.tensor([[0, 0.6], [0.3, 0.0]], device="cuda")
    keep, kept, following, err = dev([7] * 2), dev([7]), dev([7]), err_word()
    kvq.verify_runs(p, dev([0, 2]), dev([-1, 0]), u, keep, kept, following, draft=q, run_starts=dev([0, 2]), err=err)
    assert kept.item() == 1 and following.item() == 1 and err.item() == 0
    want = T.verify_runs(p.cpu().numpy(), q.cpu().numpy(), [0, 2], [-1, 0], u.cpu().numpy(), [0, 2])
    assert want[2].tolist() == [1]


@pytest.mark.parametrize("kind,status", [("nan", 6), ("inf", 6), ("negative", 7), ("above", 7), ("zeros", 7), ("random", 7), ("token", 5), ("parent", 5),
                                         ("starts", 5), ("length", 5), ("long", 5)])
def test_verification_of_what_cannot_be(kvq, kind, status):
    """Reported; the other request's path is right."""
    rng = np.random.default_rng(0)
    n0 = 3 if kind != "long" else 1025
    ns, V = [n0, 3], 50
    p = np.stack([distribution(rng, V) for _ in range(sum(ns))])
    parents = np.array(([-1, 0, 1] if n0 == 3 else [-1] + [0] * (n0 - 1)) + [-1, 0, 0])
    top = lambda r: int(np.argmax(p[r]))  # noqa: E731
    tokens = np.array([0] * n0 + [0, top(n0), 1])
    tokens[1] = top(0)
    u = np.full((sum(ns), 2), 0.5, np.float32)
    starts, lens = [0, n0, n0 + 3], [n0 + 9, 12]
    want = T.verify_runs(p[n0:], None, tokens[n0:], parents[n0:], u[n0:], [0, 3])
    t = torch.as_tensor(p).to("cuda")
    if kind in ("nan", "inf", "negative", "above"):
        t[0, 20] = {"nan": float("nan"), "inf": float("inf"), "negative": -0.5, "above": 1.5}[kind]
    elif kind == "zeros":
        t[0] = 0
    elif kind == "random":
        u[0, 1] = 1.0
    elif kind == "token":
        tokens[1] = 50
    elif kind == "parent":
        parents[1] = 2
    elif kind == "starts":
        starts = [4, 3, 6]
    elif kind == "length":
        lens = [2, 12]
    keep, kept, following, out, err = dev([7] * sum(ns)), dev([7] * 2), dev([7] * 2), dev([7] * 2), err_word()
    kvq.verify_runs(t, dev(tokens), dev(parents), dev(u, torch.float32), keep, kept, following, seq_lens=dev(lens), seq_lens_out=out, run_starts=dev(starts),
                    err=err)
    assert err.item() == status
    assert keep[n0:].tolist() == want[0].tolist() and kept[1].item() == want[1][0] and following[1].item() == want[2][0]
    assert out[1].item() == 9 + want[1][0]
    if kind in ("starts", "length", "long"):
        assert kept[0].item() == 0 and following[0].item() == -1 and out[0].item() == lens[0] and torch.all(keep[:n0] == 7)
    elif kind == "zeros":
        assert kept[0].item() == 1 and following[0].item() == -1
    elif kind == "random":
        clean = p[0].copy()
        assert following[0].item() == int(np.flatnonzero(clean)[-1]) or kept[0].item() > 1
    elif kind in ("token", "parent"):
        assert kept[0].item() == 1
    else:
        clean = p.copy()
        clean[0, 20] = 0
        want = T.verify_runs(clean[:3], None, tokens[:3], parents[:3], u[:3], [0, 3])
        assert kept[0].item() == want[1][0] and following[0].item() == want[2][0]


def test_greedy_scores_of_every_kind(kvq):
    inf, nan = float("inf"), float("nan")
    rows = [[-inf, -inf, -3.0, -inf], [-inf] * 4, [0.0, -0.0, 0.0, -1.0], [-0.0, 0.0, -1.0, -1.0], [nan, 1.0, 2.0, nan], [1.0, inf, inf, 3.0], [-1e-45, -1e-40, -1.0, -2.0]]
    want = [2, 0, 0, 0, 2, 1, 0]
    for dt in (torch.float32, torch.bfloat16):
        t = torch.tensor(rows, device="cuda").to(dt)
        keep, kept, following, err = dev([7] * 7), dev([7] * 7), dev([7] * 7), err_word()
        kvq.verify_runs(t, dev([0] * 7), dev([-1] * 7), None, keep, kept, following, err=err)
        assert following.tolist() == (want if dt is torch.float32 else want) and err.item() == 6 and kept.tolist() == [1] * 7


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("ns,V", [([129, 3, 128], 300), ([2, 64, 65, 33], 45), ([60, 4], 30011), ([5, 9], 120000), ([3] * 60, 70001)])
def test_greedy_trees_of_many_sizes(kvq, dtype, ns, V):
    verify_case(kvq, "greedy", dtype, ns, V, 5)
    verify_case(kvq, "greedy", dtype, ns, V, 6, spread=1, stride=(1, 2))


@pytest.mark.parametrize("n,V", [(6, 50), (6, 9000), (130, 50), (6, 400000)])
def test_only_scores_on_the_path_are_reported(kvq, n, V):
    """Row 0 leads to row 2; a NaN of row 1 or 3 is nobody's, one of row 2 is the path's and loses against every other score."""
    tokens, parents = [9] + [4, 7] + [7] * (n - 3), [-1, 0, 0] + [1] * (n - 3)
    for row, status in ((None, 0), (1, 0), (3, 0), (0, 6), (2, 6)):
        scores = torch.zeros((n, V), device="cuda")
        scores[0, 7], scores[2, V - 1] = 2.0, 1.0
        if row is not None:
            scores[row, V // 2 + 1] = scores[row, 0] = float("nan")
        keep, kept, following, err = dev([7] * n), dev([7]), dev([7]), err_word()
        kvq.verify_runs(scores, dev(tokens), dev(parents), None, keep, kept, following, run_starts=dev([0, n]), err=err)
        assert err.item() == status and kept.tolist() == [2] and following.tolist() == [V - 1] and keep.tolist() == [0, 2] + [-1] * (n - 2)


# ------------------------------------------------------------------------------------------------ the kept path
def keep_case(kvq, fmt, before, new, paths, heads, layers, seed=0, single=False):
    rng = np.random.default_rng(seed)
    after = np.array(before) + new
    table, pages = tables(rng, after)
    starts = starts_of(new)
    keep, kept = np.full(int(starts[-1]) + 2, -1), np.array([len(p) for p in paths])
    for s, p in enumerate(paths):
        keep[starts[s]:starts[s] + len(p)] = p
    lens = np.array(before) + kept
    caches, want = [], []
    for _ in range(layers):
        ck, cv = random_codes(rng, pages, heads, fmt), random_codes(rng, pages, heads, fmt)
        ek, ev = rng.integers(-12, -3, (pages, heads)), rng.integers(-12, -3, (pages, heads))
        caches.append(make_cache(kvq, fmt, heads, pages, ck, cv, ek, ev))
        for c, e in ((ck, ek), (cv, ev)):
            T.keep_runs(c, e, keep, kept, starts, lens, table, fmt)
        want.append((ck, cv, ek, ev))
    err = err_word()
    kvq.keep_runs(caches[0] if layers == 1 else caches, dev(lens), dev(table), dev(keep), dev(kept), run_starts=dev(starts), err=err)
    assert err.item() == 0
    for cache, w in zip(caches, want):
        check_cache(cache, fmt, heads, *w)


PATHS = [([0], [4], [[0, 2]]), ([13], [20], [[0, 4, 9, 17]]), ([13, 16, 5, 0], [20, 3, 0, 40], [[0, 4, 9, 17], [0, 1, 2], [], list(range(0, 40, 2))]),
         ([31, 1, 17], [40, 40, 40], [[39], [3, 5, 6, 8, 39], []]), ([7, 8], [16, 40], [[0], [0, 1, 2, 3, 20, 39]]), ([100], [300], [list(range(0, 300, 3))])]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("heads,layers", [(1, 1), (3, 2), (8, 5)])
@pytest.mark.parametrize("before,new,paths", PATHS)
def test_the_kept_path(kvq, fmt, heads, layers, before, new, paths):
    keep_case(kvq, fmt, before, new, paths, heads, layers)


@pytest.mark.parametrize("fmt", FMTS)
def test_the_kept_path_of_random_trees(kvq, fmt):
    rng = np.random.default_rng(8)
    for seed in range(6):
        B = int(rng.integers(1, 12))
        new = rng.integers(0, 70, B)
        paths = []
        for n in new:
            m = int(rng.integers(0, n + 1))
            paths.append(sorted(rng.choice(n, m, replace=False).tolist()))
        keep_case(kvq, fmt, rng.integers(0, 60, B), new, paths, 2, 2, seed)


def test_the_kept_path_of_more_layers_than_a_launch_takes(kvq):
    keep_case(kvq, "int8p", [3], [9], [[0, 5, 8]], 1, 131)


def test_the_largest_kept_path(kvq):
    keep_case(kvq, "e4m3p", [5], [1024], [[i for i in range(1024) if i % 50 != 7]], 1, 1)


@pytest.mark.parametrize("kind", ["not rising", "twice", "outside", "negative", "count", "negative count", "length", "page", "source page", "table", "starts"])
def test_a_path_that_cannot_be(kvq, kind):
    """Reported; that request's cache is left, the other one's moved."""
    rng = np.random.default_rng(0)
    fmt = "int8p"
    ck, cv = random_codes(rng, 8, 2, fmt), random_codes(rng, 8, 2, fmt)
    ek, ev = rng.integers(-9, -3, (8, 2)), rng.integers(-9, -3, (8, 2))
    cache = make_cache(kvq, fmt, 2, 8, ck, cv, ek, ev)
    table, starts, lens, kept = [[0, 1, 2], [3, 4, 5]], [0, 30, 40], [13, 17], [3, 2]
    keep = [-1] * 40
    keep[0:3], keep[30:32] = [0, 7, 25], [0, 4]
    if kind == "not rising":
        keep[1:3] = [25, 7]
    elif kind == "twice":
        keep[1:3] = [7, 7]
    elif kind == "outside":
        keep[2] = 30
    elif kind == "negative":
        keep[0] = -1
    elif kind == "count":
        kept[0] = 31
    elif kind == "negative count":
        kept[0] = -1
    elif kind == "length":
        lens[0] = 2
    elif kind == "page":
        table[0][0] = 8
    elif kind == "source page":
        table[0][2] = -1
    elif kind == "table":
        lens[0] = 30  # 27 + 30 tokens do not fit three pages
    else:
        starts = [31, 30, 40]
    tail = [-1] * 40
    tail[30:32] = keep[30:32]
    for c, e in ((ck, ek), (cv, ev)):
        T.keep_runs(c, e, tail, [0, 2], [0, 30, 40], [10, 17], np.array(table), fmt)
    err = err_word()
    kvq.keep_runs(cache, dev(lens), dev(table), dev(keep), dev(kept), run_starts=dev(starts), err=err)
    assert err.item() == 5
    check_cache(cache, fmt, 2, ck, cv, ek, ev)
