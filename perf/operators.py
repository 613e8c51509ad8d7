"""The serving step around a page-scaled 8-bit KV cache: page maps, quantized append and attention over it.

A page is 16 tokens; a page-scaled cache holds, for each (page, kv head), 2,048 bytes of key codes, 2,048 bytes of value
codes (E4M3, or INT8 stored as code + 128) and one power-of-two scale for each of the two.  A *run* is the new tokens that
one request brings to a step: one while it decodes, a few for a speculative draft, many for a prompt or a chunk of one.

* ``map``: lengths -> block tables, slot map, positions, free pages (``map_runs``);
* ``append``: the runs' keys and values quantized into their pages (``append_runs``);
* ``attn``: causal attention of the runs' queries over the cache (``attn_runs``).
"""
import math

import torch

own = False

PAGE, D = 16, 128
QMAX = {"e4m3p": 448.0, "int8p": 127.0}
E_MIN, E_MAX = -24, 15  # scales are powers of two that fp16 holds
DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of 64 requests around 32k tokens: one token each, a few of them open a page
        dict(name="map_decode", op="map", batch=64, lo=30000, hi=32768, new_lo=1, new_hi=1, finished=0.0, fresh=0.0),
        # a scheduler's mixed step: finished requests hand pages back, new prompts come in, the others decode
        dict(name="map_mixed", op="map", batch=256, lo=1, hi=16384, new_lo=1, new_hi=700, finished=0.1, fresh=0.2),
        # the largest map: a full batch of prompts at once
        dict(name="map_prompts", op="map", batch=1024, lo=0, hi=0, new_lo=1, new_hi=512, finished=0.0, fresh=1.0),
        # the newest token of 64 requests, 4 kv heads (the 7B-shaped INT8 workload's step)
        dict(name="append_decode_int8", op="append", batch=64, kv_heads=4, fmt="int8p", dtype="bf16", lo=2000, hi=2600,
             new_lo=1, new_hi=1),
        # a whole prompt of the cartridge workload's length, 8 kv heads
        dict(name="append_prompt_e4m3", op="append", batch=1, kv_heads=8, fmt="e4m3p", dtype="bf16", lo=0, hi=0,
             new_lo=11996, new_hi=11996),
        # chunks of odd lengths behind odd prefixes, fp32 keys
        dict(name="append_chunks_f32", op="append", batch=37, kv_heads=3, fmt="int8p", dtype="f32", lo=1, hi=1500,
             new_lo=1, new_hi=333),
        # the smallest call: one request, one token, 512 tokens of context, fp32 queries
        dict(name="attn_tiny_f32", op="attn", batch=1, kv_heads=8, q_heads=32, fmt="int8p", dtype="f32", lo=512, hi=512,
             run_lo=1, run_hi=1),
        # the 7B-shaped decode step: 64 requests of 32k tokens, 7 query heads for each kv head
        dict(name="attn_decode_int8", op="attn", batch=64, kv_heads=4, q_heads=28, fmt="int8p", dtype="bf16", lo=32768,
             hi=32768, run_lo=1, run_hi=1),
        # ragged decode of a mixed batch over pages in random order
        dict(name="attn_decode_ragged", op="attn", batch=128, kv_heads=8, q_heads=32, fmt="e4m3p", dtype="bf16", lo=1024,
             hi=16384, run_lo=1, run_hi=1),
        # speculative drafts of up to 4 tokens over the cartridge workload's length
        dict(name="attn_draft", op="attn", batch=16, kv_heads=8, q_heads=32, fmt="e4m3p", dtype="bf16", lo=11000, hi=11996,
             run_lo=2, run_hi=4),
        # chunked prefill: chunks of odd sizes beside decoding requests
        dict(name="attn_mixed", op="attn", batch=6, kv_heads=8, q_heads=32, fmt="int8p", dtype="bf16", lo=3000, hi=9001,
             run_lo=1, run_hi=1531),
        # the whole prompt of the cartridge workload's length: the largest arithmetic
        dict(name="attn_prompt", op="attn", batch=1, kv_heads=8, q_heads=32, fmt="e4m3p", dtype="bf16", lo=11996, hi=11996,
             run_lo=11996, run_hi=11996),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["map", "append", "attn", "attn"])
    fmt = rng.choice(["e4m3p", "int8p"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "map":
        batch = _log(rng, 1, 1024)
        return dict(op="map", batch=batch, lo=0, hi=_log(rng, 1, 32768), new_lo=1, new_hi=_log(rng, 1, 512),
                    finished=rng.choice([0.0, 0.1, 0.5]), fresh=rng.choice([0.0, 0.3]))
    if op == "append":
        batch = _log(rng, 1, 128)
        new = _log(rng, 1, max(1, 11996 // batch))
        return dict(op="append", batch=batch, kv_heads=rng.choice([1, 2, 3, 4, 8]), fmt=fmt, dtype=dtype, lo=rng.choice([0, 1]),
                    hi=_log(rng, 1, 2600), new_lo=max(1, new // 2), new_hi=new)
    kv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 7, 8])
    group = min(group, 32 // kv)
    kind = rng.choice(["decode", "draft", "chunk"])
    if kind == "chunk":
        # at most a quarter of the whole prompt's rows times keys, padded rows included
        batch = _log(rng, 1, 4)
        hi = _log(rng, 64, 8000)
        run = _log(rng, 1, min(hi, max(17, 30000000 // (batch * hi))))
        return dict(op="attn", batch=batch, kv_heads=kv, q_heads=kv * group, fmt=fmt, dtype="bf16", lo=max(run, hi // 2), hi=hi,
                    run_lo=max(1, run // 3), run_hi=run)
    batch = _log(rng, 1, 64)
    hi = _log(rng, 16, min(32768, 1000000 // batch))
    run = 1 if kind == "decode" else rng.choice([2, 3, 5])
    return dict(op="attn", batch=batch, kv_heads=kv, q_heads=kv * group, fmt=fmt, dtype=dtype, lo=max(run, hi // 8),
                hi=max(run, hi), run_lo=1, run_hi=run)


# ------------------------------------------------------------------------------------------------ inputs
def _lens(case, key, seed):
    """The lengths of a case: log-uniform between its bounds, the last one at the upper bound; part of the case, not of the seed's data."""
    g = torch.Generator().manual_seed(seed * 7919 + (11 if key == "run" else 5))
    names = {"len": ("lo", "hi"), "new": ("new_lo", "new_hi"), "run": ("run_lo", "run_hi")}[key]
    lo, hi = case[names[0]], case[names[1]]
    u = torch.rand(case["batch"], generator=g, dtype=torch.float64)
    a, b = math.log(max(lo, 0.5)), math.log(max(hi, 0.5) + 0.49)
    x = torch.exp(a + u * (b - a)).round().long().clamp(lo, hi)
    x[-1] = hi
    return x


def _shape(case):
    """Lengths that do not go by the seed: they set the work."""
    x = _lens(case, "len", 1)
    if case["op"] == "attn":
        return x, torch.minimum(_lens(case, "run", 2), x)
    new = _lens(case, "new", 3)
    if case["op"] == "map":
        r = torch.rand(case["batch"], generator=torch.Generator().manual_seed(17))
        x = torch.where(r < case["fresh"], torch.zeros_like(x), x)
        if 0 < case["fresh"] < 1:  # beside the new prompts the others decode
            new = torch.where(r < case["fresh"], new, torch.ones_like(new))
        if case["finished"] > 0:
            new = torch.where(r > 1 - case["finished"], torch.full_like(new, -1), new)
    return x, new


def _pages(n):
    return (n + PAGE - 1) // PAGE


def _codes_random(n, fmt, g, dev):
    """[n, 2048] bytes of codes as a normal distribution fills them."""
    out = torch.empty((n, PAGE * D), dtype=torch.uint8, device=dev)
    step = 1 << 16
    for i in range(0, n, step):
        x = torch.randn((min(step, n - i), PAGE * D), generator=g, device=dev)
        if fmt == "int8p":
            out[i:i + step] = (x * 36).round_().clamp_(-127, 127).add_(128).to(torch.uint8)
        else:
            out[i:i + step] = (x * 120).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return out


def _scales_random(heads, pages, fmt, g, dev):
    """Powers of two, fp16, head-major: about unit variance for the values that the codes stand for."""
    e = torch.randint(0, 2, (heads, pages), generator=g, device=dev) - (6 if fmt == "int8p" else 7)
    return torch.exp2(e.float()).to(torch.float16)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))
    B = case["batch"]
    st = dict(case=case, op=case["op"], err=torch.zeros(1, dtype=torch.int32, device=dev))
    i32 = dict(dtype=torch.int32, device=dev)
    lens, new = _shape(case)
    if case["op"] == "map":
        width = int(_pages(lens + new.clamp(min=0)).max()) + 1
        held = _pages(lens)
        need = int((_pages(lens + new.clamp(min=0)) - held).sum())
        total = int(held.sum()) + need + 64
        perm = torch.randperm(total, generator=g, device=dev).to(torch.int32)
        first = held.cumsum(0) - held
        at = first[:, None] + torch.arange(width)[None, :]
        mine = (torch.arange(width)[None, :] < held[:, None]).to(dev)
        bt = torch.where(mine, perm[at.clamp(max=total - 1).to(dev)], torch.full((1, 1), -1, **i32))
        nfree = total - int(held.sum())
        stack = torch.full((total,), -1, **i32)
        stack[:nfree] = perm[int(held.sum()):]
        rows = int(new.clamp(min=0).sum()) + 32  # a captured step's fixed number of rows, some of them unused
        st.update(new_lens=new.to(**i32), seq_lens=lens.to(**i32), stack=stack, count=torch.tensor([nfree], **i32), bt=bt,
                  run_starts=torch.empty(B + 1, **i32), seq_lens_out=torch.empty(B, **i32), count_out=torch.empty(1, **i32),
                  slots=torch.empty(rows, **i32), positions=torch.empty(rows, **i32))
        return st
    H, fmt = case["kv_heads"], case["fmt"]
    after = lens + new if case["op"] == "append" else lens
    n_pages = _pages(after)
    width = int(n_pages.max()) + 1
    total = int(n_pages.sum()) + 3
    perm = torch.randperm(total, generator=g, device=dev).to(torch.int32)
    first = n_pages.cumsum(0) - n_pages
    at = (first[:, None] + torch.arange(width)[None, :]).clamp(max=total - 1).to(dev)
    mine = (torch.arange(width)[None, :] < n_pages[:, None]).to(dev)
    bt = torch.where(mine, perm[at], torch.full((1, 1), -1, **i32)).contiguous()
    starts = torch.zeros(B + 1, dtype=torch.int64)
    starts[1:] = new.cumsum(0)
    rows = int(starts[-1])
    single = bool((new == 1).all())
    st.update(k=_codes_random(total * H, fmt, g, dev), v=_codes_random(total * H, fmt, g, dev),
              k_scale=_scales_random(H, total, fmt, g, dev), v_scale=_scales_random(H, total, fmt, g, dev), bt=bt,
              seq_lens=after.to(**i32), run_starts=None if single else starts.to(**i32), rows=rows, max_run=int(new.max()),
              width=width, total=total)
    dt = DTYPE[case["dtype"]]
    if case["op"] == "append":
        # keys with a few large channels, as trained models have them, so that scales grow inside a page
        kx = torch.randn((rows, H, D), generator=g, device=dev)
        kx[..., ::37] *= 6
        st.update(kx=kx.to(dt), vx=torch.randn((rows, H, D), generator=g, device=dev).to(dt))
    else:
        st.update(q=(torch.randn((rows, case["q_heads"], D), generator=g, device=dev) * 1.5).to(dt),
                  out=torch.zeros((rows, case["q_heads"], D), dtype=dt, device=dev),
                  lse=torch.zeros((rows, case["q_heads"]), device=dev))
    return st


# ------------------------------------------------------------------------------------------------ plain forms
def _unpack_k(b):
    """[..., 2048] key tiles -> [..., 16 tokens, 128 channels]."""
    s = b.shape[:-1]
    n = len(s)
    return b.view(*s, 2, 2, 8, 4, 16).permute(*range(n), n, n + 2, n + 1, n + 3, n + 4).reshape(*s, PAGE, D)


def _pack_k(x):
    s = x.shape[:-2]
    n = len(s)
    return x.reshape(*s, 2, 8, 2, 4, 16).permute(*range(n), n, n + 2, n + 1, n + 3, n + 4).reshape(*s, PAGE * D)


_V = (4, 2, 6, 0, 3, 5, 1)  # the tile's axes (c>>5, c&7, (t>>1)&3, (c>>4)&1, t>>3, (c>>3)&1, t&1) in token, channel order


def _unpack_v(b):
    s = b.shape[:-1]
    n = len(s)
    return b.view(*s, 4, 8, 4, 2, 2, 2, 2).permute(*range(n), *(n + i for i in _V)).reshape(*s, PAGE, D)


def _pack_v(x):
    s = x.shape[:-2]
    n = len(s)
    back = sorted(range(7), key=lambda i: _V[i])
    return x.reshape(*s, 2, 4, 2, 4, 2, 2, 8).permute(*range(n), *(n + i for i in back)).reshape(*s, PAGE * D)


def _values(b, fmt):
    return b.float() - 128.0 if fmt == "int8p" else b.view(torch.float8_e4m3fn).float()


def _encode(x, fmt):
    if fmt == "int8p":
        return (x.round().clamp(-127, 127) + 128.0).to(torch.uint8)
    return x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _plain_map(st):
    new, old, bt = st["new_lens"].long(), st["seq_lens"].long(), st["bt"]
    dev = bt.device
    B, width = bt.shape
    gone = new < 0
    n = new.clamp(min=0)
    held = _pages(old)
    fc = st["count"].long()
    back = torch.where(gone, held, 0)
    back_end = back.cumsum(0)
    R = back_end[-1:]
    after = torch.where(gone, 0, old + n)
    want = torch.where(gone, 0, _pages(old + n) - held)
    a_end = want.cumsum(0)
    a0 = a_end - want
    A = a_end[-1:]
    size = st["stack"].shape[0]
    # the stack with the finished requests' pages on top
    i = torch.arange(size, device=dev)
    k = i - fc
    s = torch.searchsorted(back_end, k.clamp(min=0), right=True).clamp(max=B - 1)
    j = (k - (back_end - back)[s]).clamp(0, width - 1)
    stack = torch.where((k >= 0) & (k < R), bt[s, j].long(), st["stack"].long())
    F = fc + R
    # new pages, from the top
    jj = torch.arange(width, device=dev)[None, :]
    fresh = (jj >= held[:, None]) & (jj < (held + want)[:, None])
    at = F - 1 - (a0[:, None] + jj - held[:, None])
    table = torch.where(fresh, stack[at.clamp(0, size - 1)], bt.long())
    left = F - A
    pages = torch.where(i < torch.maximum(fc, left), torch.where(i < left, stack, st["stack"].long()), st["stack"].long())
    ends = n.cumsum(0)
    starts = torch.cat([torch.zeros(1, dtype=torch.int64, device=dev), ends])
    r = torch.arange(st["slots"].shape[0], device=dev)
    seq = torch.searchsorted(ends, r, right=True).clamp(max=B - 1)
    pos = old[seq] + r - starts[seq]
    used = r < ends[-1]
    pos = torch.where(used, pos, 0)
    slot = torch.where(used, table[seq, (pos // PAGE).clamp(max=width - 1)] * PAGE + pos % PAGE, -1)
    to = lambda x: x.to(torch.int32)  # noqa: E731
    return dict(block_table=to(table), run_starts=to(starts), seq_lens=to(after), free_count=to(left), free_pages=to(pages),
                slots=to(slot), positions=to(pos))


def _starts(st):
    if st["run_starts"] is not None:
        return st["run_starts"].long()
    return torch.arange(st["bt"].shape[0] + 1, device=st["bt"].device)


def _plain_append(st):
    case, fmt = st["case"], st["case"]["fmt"]
    H, dev = case["kv_heads"], st["bt"].device
    starts, after = _starts(st), st["seq_lens"].long()
    n = starts[1:] - starts[:-1]
    first = after - n
    B, width = st["bt"].shape
    # every page that a run can touch, the absent ones masked
    m = (st["max_run"] + PAGE - 2) // PAGE + 1
    page = first[:, None] // PAGE + torch.arange(m, device=dev)[None, :]
    pos = page[..., None] * PAGE + torch.arange(PAGE, device=dev)
    fresh = (pos >= first[:, None, None]) & (pos < after[:, None, None])
    hit = fresh.any(-1)
    row = (starts[:-1, None, None] + pos - first[:, None, None]).clamp(0, st["rows"] - 1)
    phys = torch.where(hit, st["bt"].gather(1, page.clamp(max=width - 1)).long(), st["total"] - 1)
    older = (page * PAGE < first[:, None])
    keep = (pos < first[:, None, None])[:, :, None, :, None]
    is_new = fresh[:, :, None, :, None]
    for_plane = lambda p, sc, x, unpack, pack: _plain_plane(p, sc, x, unpack, pack, fmt, H, row, phys, hit, older, keep, is_new)  # noqa: E731
    for_plane(st["k"], st["k_scale"], st["kx"], _unpack_k, _pack_k)
    for_plane(st["v"], st["v_scale"], st["vx"], _unpack_v, _pack_v)
    return _append_out(st)


def _plain_plane(plane, scale, x, unpack, pack, fmt, H, row, phys, hit, older, keep, is_new):
    new = x[row].float().permute(0, 1, 3, 2, 4)  # [B, m, H, 16, 128]
    amax = torch.where(is_new, new.abs(), 0).amax((-1, -2))
    bits = amax.view(torch.int32)
    lead, k0 = (0x600000, 8) if fmt == "e4m3p" else (0x7E0000, 6)  # qmax = (1 + lead / 2^23) 2^k0
    e = ((bits >> 23) - 127 - k0 + ((bits & 0x7FFFFF) > lead).int()).clamp(E_MIN, E_MAX)
    tiles = plane.view(-1, H, PAGE * D)
    had = torch.log2(scale.t()[phys].float()).round().int()
    had = torch.where(older[..., None], had, E_MIN)
    e1 = torch.maximum(e, had)
    f = lambda k: torch.exp2(k.float())[..., None, None]  # noqa: E731
    old = _values(unpack(tiles[phys]), fmt)
    old = torch.where(keep, old * f(had - e1), 0.0)
    both = torch.where(is_new, new * f(-e1), old)
    done = hit
    tiles[phys[done]] = pack(_encode(both[done], fmt))
    scale.t()[phys[done]] = torch.exp2(e1[done].float()).to(torch.float16)


def _append_out(st):
    # the cache as it is held: codes beside their scales, both exact by definition (power-of-two scales), so they are compared
    # bit for bit, which is stricter than comparing the products of the two
    kind = torch.float8_e4m3fn if st["case"]["fmt"] == "e4m3p" else torch.uint8
    return dict(k=st["k"].view(kind), v=st["v"].view(kind), k_scale=st["k_scale"], v_scale=st["v_scale"])


def _plain_attn(st):
    case, fmt = st["case"], st["case"]["fmt"]
    B, H, Hq = case["batch"], case["kv_heads"], case["q_heads"]
    G, dev = Hq // H, st["bt"].device
    starts, lens = _starts(st), st["seq_lens"].long()
    n = starts[1:] - starts[:-1]
    N, L = st["max_run"], (st["width"] - 1) * PAGE
    pages = st["bt"][:, :st["width"] - 1].clamp(min=0).long()

    def plane(p, scale, unpack):
        x = _values(unpack(p.view(-1, H, PAGE * D)[pages]), fmt)
        x *= scale.t()[pages].float()[..., None, None]
        return x.permute(0, 2, 1, 3, 4).reshape(B, H, L, D)

    i = torch.arange(N, device=dev)
    row = (starts[:-1, None] + i).clamp(max=st["rows"] - 1)
    q = st["q"][row].float().view(B, N, H, G, D).permute(0, 2, 3, 1, 4).reshape(B, H, G * N, D)
    x = torch.matmul(q, plane(st["k"], st["k_scale"], _unpack_k).transpose(-1, -2)).view(B, H, G, N, L)
    x *= 1.0 / math.sqrt(D)
    pos = lens[:, None] - n[:, None] + i
    hidden = torch.arange(L, device=dev) > pos[..., None]
    x.masked_fill_(hidden[:, None, None], float("-inf"))
    m = x.amax(-1, keepdim=True)
    x -= m
    x.exp_()
    s = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(B, H, G * N, L), plane(st["v"], st["v_scale"], _unpack_v)).view(B, H, G, N, D) / s
    lse = (m + s.log())[..., 0]
    r = torch.arange(st["rows"], device=dev)
    seq = torch.searchsorted(starts[1:].contiguous(), r, right=True)
    off = r - starts[seq]
    st["out"].copy_(o.permute(0, 3, 1, 2, 4)[seq, off].reshape(-1, Hq, D))
    st["lse"].copy_(lse.permute(0, 3, 1, 2)[seq, off].reshape(-1, Hq))
    return dict(out=st["out"], lse=st["lse"])


# ------------------------------------------------------------------------------------------------ the framework's operators
def _own(st):
    import quantized_kv_cache_kvq_gb300 as kvq

    case = st["case"]
    if st["op"] == "map":
        kvq.map_runs(st["new_lens"], st["seq_lens"], st["stack"], st["count"], st["bt"], st["run_starts"], st["seq_lens_out"],
                     st["count_out"], slot_mapping=st["slots"], positions=st["positions"], err=st["err"])
        return dict(block_table=st["bt"], run_starts=st["run_starts"], seq_lens=st["seq_lens_out"], free_count=st["count_out"],
                    free_pages=st["stack"], slots=st["slots"], positions=st["positions"])
    if "cache" not in st:
        st["cache"] = kvq.PagedCache.over(case["fmt"], case["fmt"], case["kv_heads"], st["total"], k=st["k"], v=st["v"],
                                          k_scale=st["k_scale"], v_scale=st["v_scale"])
    if st["op"] == "append":
        kvq.append_runs(st["cache"], st["kx"], st["vx"], st["seq_lens"], st["bt"], run_starts=st["run_starts"], err=st["err"])
        return _append_out(st)
    if "workspace" not in st:
        st["workspace"] = torch.empty(kvq.attn_runs_workspace_size(case["batch"], st["rows"], st["max_run"], case["kv_heads"],
                                                                   case["q_heads"], st["q"].dtype),
                                      dtype=torch.uint8, device=st["q"].device)
    kvq.attn_runs(st["cache"], st["q"], st["seq_lens"], st["bt"], st["out"], st["workspace"], run_starts=st["run_starts"],
                  max_run=st["max_run"], lse=st["lse"], err=st["err"])
    return dict(out=st["out"], lse=st["lse"])


def run(state):
    if own:
        return _own(state)
    if state["op"] == "map":
        return _plain_map(state)
    if state["op"] == "append":
        return _plain_append(state)
    return _plain_attn(state)


# ------------------------------------------------------------------------------------------------ work
def work(case):
    lens, new = _shape(case)
    B = case["batch"]
    if case["op"] == "map":
        n = new.clamp(min=0)
        pages = int((_pages(lens + n) - _pages(lens)).sum()) + int(_pages(lens)[new < 0].sum())
        return {"bytes": 16 * B + 12 + 8 * int(n.sum()) + 8 * pages, "flops": 0}
    size = 2 if case["dtype"] == "bf16" else 4
    H = case["kv_heads"]
    if case["op"] == "append":
        n = int(new.sum())
        return {"bytes": 2 * n * H * D * (size + 1) + 4 * H * (n / PAGE + B), "flops": 6 * n * H * D}
    Hq = case["q_heads"]
    rows = int(new.sum())
    seen = float((new * lens - new * (new - 1) // 2).sum())  # (row, key) pairs under the causal mask
    keys = int(lens.sum())
    return {"bytes": 2 * keys * H * D + 4 * H * keys / PAGE + rows * Hq * (2 * D * size + 4), "flops": 4.0 * D * Hq * seen}


# ------------------------------------------------------------------------------------------------ in 64 bits
def _tile_order():
    """Byte of (token, channel) in a key tile and in a value tile."""
    t, c = torch.arange(PAGE)[:, None], torch.arange(D)[None, :]
    k = 16 * (((t >> 3) * 2 + (c >> 6)) * 32 + (t & 7) * 4 + ((c >> 4) & 3)) + (c & 15)
    v = 16 * (32 * (c >> 5) + 4 * (c & 7) + ((t & 7) >> 1)) + 8 * ((c >> 4) & 1) + 2 * (2 * (t >> 3) + ((c >> 3) & 1)) + (t & 1)
    return k.reshape(-1), v.reshape(-1)


def _float_of_e4m3(b):
    b = b.to(torch.int64)
    e, m = (b >> 3) & 15, (b & 7).double()
    x = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.exp2((e - 10).double()))
    return torch.where(b >= 128, -x, x)


def exact(case, seed):
    if case["op"] == "map":
        return None
    st = prepare(case, seed)
    fmt, H = case["fmt"], case["kv_heads"]
    dev = st["bt"].device
    ko, vo = (o.to(dev) for o in _tile_order())
    value = (lambda b: b.double() - 128) if fmt == "int8p" else _float_of_e4m3
    starts, lens = _starts(st).tolist(), st["seq_lens"].tolist()
    if case["op"] == "append":
        q = QMAX[fmt]
        grid = _float_of_e4m3(torch.arange(127, device=dev)) if fmt == "e4m3p" else torch.arange(128, device=dev, dtype=torch.float64)

        def nearest(x):  # the nearest value of the grid, ties to the even code
            a = x.abs().clamp(max=float(grid[-1])).contiguous()
            hi = torch.searchsorted(grid, a).clamp(max=len(grid) - 1)
            lo = (hi - 1).clamp(min=0)
            up, down = grid[hi] - a, a - grid[lo]
            pick = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
            return torch.copysign(grid[pick], x)

        outs = {}
        for name, order, x in (("k", ko, st["kx"]), ("v", vo, st["vx"])):
            tiles, scale = st[name].view(-1, H, PAGE * D), st[name + "_scale"]
            codes = value(tiles)  # by byte of the tile
            for s in range(case["batch"]):
                n = starts[s + 1] - starts[s]
                first = lens[s] - n
                for page in range(first // PAGE, _pages(lens[s])):
                    phys = int(st["bt"][s, page])
                    p0 = page * PAGE
                    lo, hi = max(first, p0), min(lens[s], p0 + PAGE)
                    new = x[starts[s] + lo - first:starts[s] + hi - first].double().permute(1, 0, 2)  # [H, n, D]
                    top = new.abs().amax((1, 2))
                    e = torch.ceil(torch.log2((top / q).clamp(min=2.0 ** -60)))
                    e = torch.where(top > q * torch.exp2(e), e + 1, e)
                    e = torch.where(top <= q * torch.exp2(e - 1), e - 1, e).clamp(E_MIN, E_MAX)
                    had = torch.log2(scale[:, phys].double()).round() if lo > p0 else torch.full_like(e, E_MIN)
                    e1 = torch.maximum(e, had)
                    page_codes = torch.zeros((H, PAGE, D), dtype=torch.float64, device=dev)
                    if lo > p0:
                        was = codes[phys][:, order].view(H, PAGE, D)[:, :lo - p0]
                        page_codes[:, :lo - p0] = nearest(was * torch.exp2(had - e1)[:, None, None])
                    page_codes[:, lo - p0:hi - p0] = nearest(new * torch.exp2(-e1)[:, None, None])
                    codes[phys][:, order] = page_codes.view(H, -1)
                    scale[:, phys] = torch.exp2(e1).to(torch.float16)
            # INT8 comes back as its bytes: whole numbers, nothing to measure in 64 bits
            outs[name] = codes.view(st[name].shape) if fmt == "e4m3p" else None
            outs[name + "_scale"] = scale.double()
        return outs
    Hq = case["q_heads"]
    G = Hq // H
    if 4.0 * D * Hq * sum((starts[s + 1] - starts[s]) * lens[s] for s in range(case["batch"])) > 6e12:
        return None
    out = torch.zeros((st["rows"], Hq, D), dtype=torch.float64, device=dev)
    lse = torch.zeros((st["rows"], Hq), dtype=torch.float64, device=dev)
    for s in range(case["batch"]):
        n = starts[s + 1] - starts[s]
        pages = st["bt"][s, :_pages(lens[s])].long()
        for h in range(H):
            k, v = ((value(st[p].view(-1, H, PAGE * D)[pages, h][:, o]) * st[p + "_scale"][h, pages].double()[:, None])
                    .view(-1, D)[:lens[s]] for p, o in (("k", ko), ("v", vo)))
            for i0 in range(0, n, 2048):
                i1 = min(n, i0 + 2048)
                last = lens[s] - n + i1
                seen = torch.arange(last, device=dev)[None, :] <= (lens[s] - n + torch.arange(i0, i1, device=dev))[:, None]
                q = st["q"][starts[s] + i0:starts[s] + i1, h * G:(h + 1) * G].double()
                x = torch.einsum("igd,td->igt", q, k[:last]) / math.sqrt(D)
                x = torch.where(seen[:, None, :], x, -math.inf)
                z = torch.logsumexp(x, -1)
                at = slice(starts[s] + i0, starts[s] + i1)
                out[at, h * G:(h + 1) * G] = torch.einsum("igt,td->igd", torch.exp(x - z[..., None]), v[:last])
                lse[at, h * G:(h + 1) * G] = z
    return dict(out=out, lse=lse)
