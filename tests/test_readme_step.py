"""The step of many requests that README.md shows: what it passes (CPU), and that a step which is refused is seen (GPU)."""
import os
import re
import types

import pytest

torch = pytest.importorskip("torch")

README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def step():
    blocks = [b for b in re.findall(r"```python\n(.*?)```", open(README).read(), flags=re.S) if "map_runs(" in b]
    assert len(blocks) == 1
    return blocks[0]


def test_every_call_reports_and_the_map_knows_the_rows():
    calls = {}
    kvq = types.SimpleNamespace(PagedCache=lambda *a: None, attn_runs_workspace_size=lambda *a: 1,
                                **{n: (lambda *a, n=n, **kw: calls.__setitem__(n, kw)) for n in ("map_runs", "append_runs", "attn_runs")})
    names = {n: 1 for n in "num_kv_heads num_pages num_q_heads B rows max_run new_lens seq_lens free_pages free_count block_table "
             "run_starts k v out".split()}
    fake_torch = types.SimpleNamespace(empty=lambda *a, **kw: None, zeros=lambda *a, **kw: "err", uint8=None, int32=None)
    exec(step(), dict(names, kvq=kvq, torch=fake_torch, q=types.SimpleNamespace(dtype=None)))
    assert all(calls[n]["err"] == "err" for n in ("map_runs", "append_runs", "attn_runs"))
    assert calls["map_runs"]["max_rows"] == names["rows"] and calls["attn_runs"]["max_run"] == names["max_run"]


@pytest.mark.gpu
@pytest.mark.parametrize("new,pages,status", [([20, 5], 4, 0), ([20, 40], 4, 9), ([20, 33], 9, 5)])
def test_a_step_that_is_refused_is_seen_in_err(new, pages, status):
    import quantized_kv_cache_kvq_gb300 as kvq

    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    rows = 48 if status != 9 else 64
    env = dict(kvq=kvq, torch=torch, num_kv_heads=1, num_q_heads=2, num_pages=pages, B=2, rows=rows, max_run=rows, new_lens=i32(*new),
               seq_lens=i32(0, 0), free_pages=torch.arange(pages, dtype=torch.int32, device="cuda"), free_count=i32(pages),
               block_table=torch.full((2, 4), -1, dtype=torch.int32, device="cuda"), run_starts=i32(0, 0, 0))
    x = torch.randn(rows, 4, 128, device="cuda").bfloat16()
    env.update(q=x[:, :2], k=x[:, 2:3], v=x[:, 3:], out=torch.full((rows, 2, 128), 7.0, device="cuda").bfloat16())
    exec(step(), env)
    assert kvq.read_err(env["err"]) == status
    taken = sum(new) if status == 0 else 0
    assert env["seq_lens"].tolist() == (new if taken else [0, 0]) and env["run_starts"].tolist()[-1] == taken
    assert torch.all(env["out"][taken:] == 7) and not torch.any(torch.all(env["out"][:taken] == 7, -1))
