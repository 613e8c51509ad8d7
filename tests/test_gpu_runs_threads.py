"""The runs' calls from two host threads, each with its own stream, batch and cache (GPU)."""
import threading

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def job(kvq, fmt, batch, dtype, max_run, seed):
    """Buffers of one step: map, append, attention; returns (step(stream), outputs)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    H, G, width = 2, 4, 4
    pages = batch * width
    i32 = dict(dtype=torch.int32, device="cuda")
    new = torch.randint(1, max_run + 1, (batch,), generator=g, **i32)
    rows = int(new.sum())
    x = torch.randn(rows, H * G + 2 * H, 128, generator=g, device="cuda").to(dtype)
    cache = kvq.PagedCache(fmt, fmt, H, pages)
    stack, count = torch.arange(pages, **i32), torch.tensor([pages], **i32)
    table, lens, starts = torch.full((batch, width), -1, **i32), torch.zeros(batch, **i32), torch.zeros(batch + 1, **i32)
    out, err = torch.zeros(rows, H * G, 128, dtype=dtype, device="cuda"), torch.zeros(1, **i32)
    ws = torch.empty(kvq.attn_runs_workspace_size(batch, rows, max_run, H, H * G, dtype), dtype=torch.uint8, device="cuda")

    def step(stream):
        table.fill_(-1)
        lens.zero_()
        count.fill_(pages)
        stack.copy_(torch.arange(pages, **i32))
        out.zero_()
        kvq.map_runs(new, lens, stack, count, table, starts, lens, count, max_rows=rows, err=err, stream=stream)
        kvq.append_runs(cache, x[:, H * G:H * G + H], x[:, H * G + H:], lens, table, run_starts=starts, err=err, stream=stream)
        kvq.attn_runs(cache, x[:, :H * G], lens, table, out, ws, run_starts=starts, max_run=max_run, err=err, stream=stream)
        return out.clone(), cache.k.clone(), err.clone()

    return step


@pytest.mark.parametrize("dtype,max_run", [(torch.bfloat16, 1), (torch.bfloat16, 4), (torch.bfloat16, 40), (torch.float32, 5)])
def test_two_threads_with_batches_of_their_own(dtype, max_run):
    import quantized_kv_cache_kvq_gb300 as kvq

    kvq.load()
    jobs = [job(kvq, "int8p", 1, dtype, max_run, 1), job(kvq, "int8p", 700, dtype, max_run, 2)]
    torch.cuda.synchronize()
    got, faults, barrier = [[], []], [], threading.Barrier(2)

    def work(i):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                barrier.wait(timeout=30)
                for _ in range(10):
                    got[i].append(jobs[i](stream))
            stream.synchronize()
        except Exception as e:  # noqa: BLE001
            faults.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not faults, faults
    for i in range(2):
        want = jobs[i](None)
        torch.cuda.synchronize()
        assert want[2].item() == 0
        for one in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(one, want))
