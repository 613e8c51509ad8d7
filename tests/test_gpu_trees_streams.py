"""The calls for trees on a stream of their own (GPU), while the default stream is held: one that is queued anywhere else has not run when its
results are looked at."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from oracle import trees as T  # noqa: E402
from tests.runs_cases import random_codes, starts_of, tables  # noqa: E402
from tests.test_gpu_runs import dev, err_word, make_cache  # noqa: E402
from tests.tree_cases import distribution, random_trees  # noqa: E402


@pytest.fixture(scope="module")
def kvq():
    import quantized_kv_cache_kvq_gb300 as m

    m.load()
    return m


@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("ns,dtype", [([40, 33], torch.bfloat16), ([3, 2], torch.bfloat16), ([9, 4], torch.float32)])
def test_every_call_runs_on_its_stream(kvq, given, ns, dtype):
    """``given``: the stream as an argument, beside a current stream that is another one."""
    rng = np.random.default_rng(sum(ns))
    H, Hq, V = 2, 8, 50
    rows, starts, lens = sum(ns), starts_of(ns), np.array([90, 60])
    parents = random_trees(rng, ns, 3)
    want_mask, want_pos = T.tree_runs(parents, starts, lens, 2)
    table, pages = tables(rng, lens)
    codes, e = random_codes(rng, pages, H, "int8p"), rng.integers(-8, -4, (pages, H))
    p, q = (np.stack([distribution(rng, V) for _ in range(rows)]) for _ in range(2))
    tokens, u = rng.integers(0, V, rows), rng.random((rows, 2)).astype(np.float32)
    walk = T.verify_runs(p, q, tokens, parents, u, starts)
    forced, forced_kept = np.full(rows, -1), [2, 1]
    forced[:2], forced[ns[0]] = [0, ns[0] - 1], 0
    stream = torch.cuda.Stream()
    on = dict(stream=stream) if given else {}
    results = []

    def calls():
        """All five, into outputs that this stream clears just before."""
        mask, positions, keep, kept, following = state["mask"], state["positions"], state["keep"], state["kept"], state["next"]
        with torch.cuda.stream(stream):
            for t in (mask, positions, keep, kept, following, state["out"], state["y"], state["err"]):
                t.zero_()
            for plane, t in state["planes"].items():  # keep_runs moves tokens
                getattr(state["cache"], plane).copy_(t)
        with torch.cuda.stream(torch.cuda.default_stream() if given else stream):
            run = dict(run_starts=state["starts"], err=state["err"], **on)
            kvq.tree_runs(state["parents"], state["lens"], mask, positions=positions, **run)
            kvq.rope_runs(state["x"], None, positions, state["cs"], q_out=state["y"], **run)
            kvq.attn_tree(state["cache"], state["x"], state["lens"], state["table"], mask, state["out"], state["ws"], max_run=max(ns), **run)
            kvq.verify_runs(state["p"], state["tokens"], state["parents"], state["u"], keep, kept, following, draft=state["q"], **run)
            kvq.keep_runs(state["cache"], state["kept_to"], state["table"], state["forced"], state["forced_kept"], **run)
        with torch.cuda.stream(stream):
            got = [t.cpu() for t in (mask, positions, state["y"], state["out"], keep, kept, following, state["cache"].k, state["err"])]
        stream.synchronize()
        results.append(got)

    with torch.cuda.stream(stream):
        state = dict(parents=dev(parents), lens=dev(lens), table=dev(table), starts=dev(starts), tokens=dev(tokens), u=dev(u, torch.float32),
                     p=dev(p, torch.float32), q=dev(q, torch.float32), forced=dev(forced), forced_kept=dev(forced_kept),
                     kept_to=dev(lens - np.array(ns) + forced_kept), mask=dev(np.zeros((rows, 2))), positions=dev(np.zeros(rows)), keep=dev(np.zeros(rows)),
                     kept=dev([0, 0]), next=dev([0, 0]), err=err_word(), x=torch.randn((rows, Hq, 128), device="cuda").to(dtype),
                     cs=torch.randn((100, 128), device="cuda"), cache=make_cache(kvq, "int8p", H, pages, codes, codes, e, e))
        state["y"], state["out"] = torch.zeros_like(state["x"]), torch.zeros_like(state["x"])
        state["ws"] = torch.empty(kvq.attn_tree_workspace_size(2, rows, max(ns), H, Hq, dtype), dtype=torch.uint8, device="cuda")
        state["planes"] = {plane: getattr(state["cache"], plane).clone() for plane in ("k", "v", "k_scale", "v_scale")}
    torch.cuda.synchronize()
    calls()  # kernels are loaded, allocations made
    torch.cuda.synchronize()
    torch.cuda._sleep(1_000_000_000)  # half a second of the default stream
    behind = torch.cuda.Event()
    behind.record()
    calls()
    assert not behind.query(), "the default stream was through before the results were read"
    torch.cuda.synchronize()
    mask, positions, y, out, keep, kept, following, k, err = results[1]
    assert err.item() == 0
    assert np.array_equal(mask.numpy(), want_mask) and np.array_equal(positions.numpy(), want_pos)
    exact = T.rope(state["x"].double().cpu().numpy(), None, 0.0, want_pos, state["cs"].double().cpu().numpy())
    # two products of values below 8 and below 8, binary32; rounded to the output's type
    assert np.all(np.abs(y.double().numpy() - exact) <= 2.0 ** -22 * 128 + (2.0 ** -8 if dtype is torch.bfloat16 else 2.0 ** -24) * np.abs(exact))
    assert keep.tolist() == walk[0].tolist() and kept.tolist() == walk[1].tolist() and following.tolist() == walk[2].tolist()
    assert torch.all(torch.any(out != 0, -1)) and not torch.equal(k, state["planes"]["k"].cpu())
    for a, b in zip(*results):  # and what they gave when nothing was held
        assert torch.equal(a, b)
