"""Operators over a 4-bit (q4_0) paged KV cache and device-built block tables:
cases, plain torch forms and the library's calls.

Four operators:

* ``write``   -- the slot write into a q4_0 pool (quantizing 32 values to one
  fp16 scale and 4-bit codes) and the read-back of the written rows;
* ``decode``  -- decode attention over a q4_0 pool, one query token a
  sequence, plain or through a sharing-aware plan;
* ``prefill`` -- chunked-prefill attention over a q4_0 pool;
* ``tables``  -- block tables, slot map, positions and lengths of a batch
  built from the requests' token counts and a ring of free blocks.

Pool layout: uint8 ``[L, N, H_kv, B * D / 2 + B * D / 16]``; a (block, head)
chunk holds D / 32 code planes ``[B][16 bytes]`` (value 2i of a group in the
low nibble of byte i, 2i + 1 in the high one, code c as c + 8), then the fp16
scales, ``[B][D / 32]`` in the K pool and ``[D / 32][B]`` in the V pool.
"""

import math

import numpy as np
import torch

own = False

DEV = "cuda"


# --------------------------------------------------------------------- cases


def listed():
    return [
        # -- slot write and read-back
        # one decode step of a 37-sequence batch, one layer: latency
        dict(name="write_step37", op="write", L=1, n=37, N=5461, B=16, H=8, D=128),
        # one decode step of 128 sequences written to all 36 layers at once
        dict(name="write_step128_36l", op="write", L=36, n=128, N=512, B=16, H=8, D=128),
        # a 4097-token prefill round into one layer, small heads, blocks of 8
        dict(name="write_chunk4097_d64", op="write", L=1, n=4097, N=2048, B=8, H=6, D=64),
        # -- decode
        # one short sequence, a handful of query heads: latency
        dict(name="decode_333", op="decode", N=64, B=16, H=4, G=4, D=128, n_par=1, n_br=1, lo=333, hi=333),
        # 37 independent sequences around 2K tokens, 32 query and 8 K/V heads
        dict(name="decode_37x2k", op="decode", N=5461, B=16, H=8, G=4, D=128, n_par=37, n_br=1, lo=2048, hi=2303),
        # one sequence of 131,071 tokens: the split over a long axis
        dict(name="decode_131071", op="decode", N=4200, B=32, H=8, G=8, D=128, n_par=1, n_br=1, lo=131071, hi=131071),
        # 12 parents of 32,771 tokens, four branches each, 64 query heads: shared blocks read once
        dict(name="decode_shared_32k", op="decode", N=25600, B=16, H=8, G=8, D=128, n_par=12, n_br=4, lo=32771, hi=32771),
        # -- chunked prefill
        # three short chunks after histories of 0, 37 and 200 tokens
        dict(name="prefill_tiny", op="prefill", N=64, B=16, H=2, G=4, D=128, hist="0,37,200", chunk="45,130,1"),
        # a 4096-token round: eight 512-token chunks after histories of 0 to 7680 tokens
        dict(name="prefill_8x512", op="prefill", N=2304, B=16, H=8, G=4, D=128,
             hist="0,512,1536,2560,3584,4608,5632,7680", chunk="512,512,512,512,512,512,512,512"),
        # -- block tables
        # one decode step of 37 sequences around 2K tokens: latency
        dict(name="tables_step37", op="tables", B=16, rows=64, n=37, mb=256, lo=2047, hi=2302, clo=1, chi=1),
        # one decode step of 1000 sequences of up to 32K tokens
        dict(name="tables_step1000", op="tables", B=16, rows=1024, n=1000, mb=2050, lo=255, hi=32767, clo=1, chi=1),
        # admission of 67 prompts, 131K new tokens in all
        dict(name="tables_admit67", op="tables", B=16, rows=128, n=67, mb=512, lo=0, hi=3, clo=17, chi=3900),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "decode", "decode", "prefill", "tables"])
    if op == "write":
        L = rng.choice([1, 1, 2, 36])
        n = _log(rng, 1, 4000 // L if L > 2 else 4000)
        return dict(op=op, L=L, n=n, N=rng.randint(600, 900), B=rng.choice([8, 16, 32, 64]), H=rng.choice([1, 2, 4, 6, 8]),
                    D=rng.choice([64, 128]))
    if op == "decode":
        B, H, G = rng.choice([8, 16, 32, 64, 128]), rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 8])
        n_br = rng.choice([1, 1, 3])
        total = _log(rng, 40, 200000)
        n_par = min(_log(rng, 1, 128), max(1, total // 20))
        mean = max(2, total // n_par)
        lo, hi = max(1, mean // 2), mean + mean // 2
        N = n_par * (hi // B + 2) + n_par * n_br + 5
        return dict(op=op, N=N, B=B, H=H, G=G, D=rng.choice([64, 128]), n_par=n_par, n_br=n_br, lo=lo, hi=hi)
    if op == "prefill":
        n, B = rng.randint(1, 4), rng.choice([8, 16, 32, 64])
        hist = [0 if rng.random() < 0.2 else _log(rng, 1, 4000) for _ in range(n)]
        chunk = [_log(rng, 1, 400) for _ in range(n)]
        N = sum(-(-(h + c) // B) for h, c in zip(hist, chunk)) + 7
        return dict(op=op, N=N, B=B, H=rng.choice([1, 2, 4, 8]), G=rng.choice([1, 2, 4, 8]), D=128,
                    hist=",".join(map(str, hist)), chunk=",".join(map(str, chunk)))
    n, B = _log(rng, 1, 1000), rng.choice([8, 16, 32, 64])
    hi = _log(rng, 20, 15000)
    chi = rng.choice([1, 1, 4, _log(rng, 4, max(5, 100000 // n))])
    return dict(op="tables", B=B, rows=n + rng.randint(0, 40), n=n, mb=-(-(hi + chi) // B) + rng.randint(0, 9),
                lo=0, hi=hi, clo=0 if chi > 1 else 1, chi=chi)


# -------------------------------------------------- host facts of a case


def _ints(text):
    return [int(x) for x in text.split(",")]


def _lens(case):
    """Parents' context lengths (before the branch's own token), from the case alone."""
    r = np.random.RandomState(case["n_par"] * 7 + case["lo"] % 1000)
    return r.randint(case["lo"], case["hi"] + 1, case["n_par"])


def _batch(case, perm):
    """Block table rows and context lengths of a decode batch.  n_br == 1: the
    parents themselves.  Else every parent is forked n_br times, stays alive,
    and each branch appends one token: a branch's partly filled last block is
    its own copy, the full blocks are the parent's."""
    B, ids, rows, lens = case["B"], iter(perm.tolist()), [], []
    tables = [[next(ids) for _ in range(-(-int(c) // B))] for c in _lens(case)]
    for t, c in zip(tables, _lens(case)):
        if case["n_br"] == 1:
            rows.append(t)
            lens.append(int(c))
        for _ in range(case["n_br"] if case["n_br"] > 1 else 0):
            rows.append(t[: int(c) // B] + [next(ids)])
            lens.append(int(c) + 1)
    mb = max(len(r) for r in rows)
    table = np.full((len(rows), mb), -1, dtype=np.int32)
    for i, r in enumerate(rows):
        table[i, : len(r)] = r
    return table, np.array(lens, dtype=np.int32)


def _counts(case):
    r = np.random.RandomState(case["n"] + case["mb"])
    old = r.randint(case["lo"], case["hi"] + 1, case["n"])
    return old.astype(np.int32), r.randint(case["clo"], case["chi"] + 1, case["n"]).astype(np.int32)


# ----------------------------------------------------------- q4_0 in torch


def _quantize(x):
    """float32 [..., 32] -> codes + 8 (uint8), fp16 scales [...]."""
    d = (x.abs().amax(-1) / 7).half()
    df = d.float().unsqueeze(-1)
    q = torch.where(df > 0, torch.round(x / df), torch.zeros_like(x))
    return (q.clamp(-7, 7) + 8).to(torch.uint8), d


def _nibbles(code):
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _parts(pool, B, D, name):
    """Views of a pool [L, N, H, chunk]: codes [L, N, H, D/32, B, 16], scales [L, N, H, B, D/32]."""
    codes = pool[..., : B * D // 2].unflatten(-1, (D // 32, B, 16))
    scales = pool[..., B * D // 2 :].view(torch.float16)
    if name == "k":
        return codes, scales.unflatten(-1, (B, D // 32))
    return codes, scales.unflatten(-1, (D // 32, B)).transpose(-1, -2)


def _values(codes, scales):
    """Codes [..., 16] and scales [...] -> float32 [..., 32]."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    return (c.float() - 8) * scales.float().unsqueeze(-1)


def _fill(N, B, H, D, g, name):
    """A pool of one layer holding quantized N(0, 1) rows."""
    pool = torch.empty(1, N, H, B * D // 2 + B * D // 16, dtype=torch.uint8, device=DEV)
    codes, scales = _parts(pool, B, D, name)
    for a in range(0, N, 2048):
        b = min(N, a + 2048)
        x = torch.randn(b - a, H, D // 32, B, 32, device=DEV, generator=g).bfloat16().float()
        q, d = _quantize(x)
        codes[0, a:b] = _nibbles(q)
        scales[0, a:b] = d.transpose(2, 3)
    return pool


# ------------------------------------------------------------------- prepare


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 9973 + 17)
    r = np.random.RandomState(seed % (1 << 31))
    return {"write": _prep_write, "decode": _prep_decode, "prefill": _prep_prefill,
            "tables": _prep_tables}[case["op"]](case, g, r)


def _bf16(g, *shape):
    return torch.randn(*shape, device=DEV, generator=g).bfloat16()


def _cache(case, k, v, free_order=None):
    from paged_kv_cache_65_gb300 import PagedKVCache

    return PagedKVCache(k.shape[0], case["N"], case["B"], case["H"], case["D"], "q4_0", k_cache=k, v_cache=v,
                        free_order=free_order)


def _prep_write(case, g, r):
    L, n, N, B, H, D = (case[x] for x in ("L", "n", "N", "B", "H", "D"))
    shape = (L, N, H, B * D // 2 + B * D // 16)
    s = dict(case=case, k_pool=torch.zeros(shape, dtype=torch.uint8, device=DEV),
             v_pool=torch.zeros(shape, dtype=torch.uint8, device=DEV),
             k=_bf16(g, L, n, H, D), v=_bf16(g, L, n, H, D),
             slots=torch.from_numpy(r.permutation(N * B)[:n].astype(np.int64)).to(DEV),
             k_out=torch.zeros(L, n, H, D, device=DEV), v_out=torch.zeros(L, n, H, D, device=DEV))
    if own:
        s["cache"] = _cache(case, s["k_pool"], s["v_pool"])
    return s


def _prep_decode(case, g, r):
    N, B, H, G, D = (case[x] for x in ("N", "B", "H", "G", "D"))
    perm = r.permutation(N).astype(np.int32)
    table, lens = _batch(case, perm)
    n, mb = table.shape
    s = dict(case=case, k_pool=_fill(N, B, H, D, g, "k"), v_pool=_fill(N, B, H, D, g, "v"), q=_bf16(g, n, H * G, D),
             table=torch.from_numpy(table).to(DEV), lens=torch.from_numpy(lens).to(DEV), n=n, mb=mb,
             out=torch.empty(n, H * G, D, dtype=torch.bfloat16, device=DEV))
    if own:
        c = s["cache"] = _cache(case, s["k_pool"], s["v_pool"], free_order=perm)
        if case["n_br"] > 1:  # the manager's sequences, for the plan
            for i, length in enumerate(_lens(case)):
                c.seq_append_tokens(100000 + i, int(length))
            for i in range(n):
                c.seq_fork(100000 + i // case["n_br"], i)
            c.seq_append_slots(list(range(n)))
            mine, _ = c.seq_block_table(list(range(n)), mb)
            assert (mine == table).all()
            s["h_plan"], ws = c.paged_decode_plan(list(range(n)), H * G, mb)
            s["d_plan"] = torch.from_numpy(s["h_plan"]).to(DEV)
        else:
            ws = c.paged_decode_workspace_bytes(n, H * G)
        s["ws"] = torch.empty(ws, dtype=torch.uint8, device=DEV)
    return s


def _prep_prefill(case, g, r):
    N, B, H, G, D = (case[x] for x in ("N", "B", "H", "G", "D"))
    hist, chunk = _ints(case["hist"]), _ints(case["chunk"])
    perm, at, n = r.permutation(N).astype(np.int32), 0, len(hist)
    mb = max(-(-(h + c) // B) for h, c in zip(hist, chunk))
    table = np.full((n, mb), -1, dtype=np.int32)
    for i, (h, c) in enumerate(zip(hist, chunk)):
        k = -(-(h + c) // B)
        table[i, :k] = perm[at : at + k]
        at += k
    start = np.concatenate([[0], np.cumsum(chunk)]).astype(np.int32)
    lens = (np.array(hist) + np.array(chunk)).astype(np.int32)
    s = dict(case=case, k_pool=_fill(N, B, H, D, g, "k"), v_pool=_fill(N, B, H, D, g, "v"),
             q=_bf16(g, int(start[-1]), H * G, D),
             table=torch.from_numpy(table).to(DEV), lens=torch.from_numpy(lens).to(DEV), n=n, mb=mb,
             start=torch.from_numpy(start).to(DEV), max_chunk=max(chunk),
             out=torch.empty(int(start[-1]), H * G, D, dtype=torch.bfloat16, device=DEV))
    if own:
        c = s["cache"] = _cache(case, s["k_pool"], s["v_pool"])
        s["ws"] = torch.empty(c.paged_prefill_staging_bytes(n, mb), dtype=torch.uint8, device=DEV)
        sched = c.paged_prefill_schedule(start, lens, H * G)
        s["sched"], s["n_items"] = torch.from_numpy(sched).to(DEV), len(sched)
    return s


def _prep_tables(case, g, r):
    B, R, n, mb = (case[x] for x in ("B", "rows", "n", "mb"))
    old, cnt = _counts(case)
    rows = r.permutation(R)[:n].astype(np.int32)
    have = -(-old // B)
    N = int(have.sum() + (-(-(old + cnt) // B) - have).sum()) + 64
    perm = r.permutation(N).astype(np.int32)
    tables = np.full((R, mb), -1, dtype=np.int32)
    lens = np.zeros(R, dtype=np.int32)
    lens[rows] = old
    at = 0
    for i in range(n):
        tables[rows[i], : have[i]] = perm[at : at + have[i]]
        at += have[i]
    # the free blocks in a ring of N entries, the oldest one somewhere inside it
    head, count = int(r.randint(N)), N - at
    ring = np.full(N, -1, dtype=np.int32)
    ring[(head + np.arange(count)) % N] = perm[at:]
    T = int(cnt.sum()) + 5  # a padded token count
    i32 = dict(dtype=torch.int32, device=DEV)
    s = dict(case=case, tables=torch.from_numpy(tables).to(DEV), lens=torch.from_numpy(lens).to(DEV),
             ring=torch.from_numpy(ring).to(DEV), state=torch.tensor([head, count], dtype=torch.int64, device=DEV),
             rows=torch.from_numpy(rows).to(DEV), counts=torch.from_numpy(cnt).to(DEV), T=T,
             slots=torch.empty(T, dtype=torch.int64, device=DEV), positions=torch.empty(T, **i32),
             start=torch.empty(n + 1, **i32), block_table=torch.empty(n, mb, **i32), context=torch.empty(n, **i32),
             lens_out=torch.empty(R, **i32), state_out=torch.empty(2, dtype=torch.int64, device=DEV))
    if own:
        from paged_kv_cache_65_gb300 import PagedKVCache
        from paged_kv_cache_65_gb300.cache import DeviceTables

        c = s["cache"] = PagedKVCache(1, N, B, 1, 64, "bf16")
        s["dt"] = DeviceTables(s["tables"], s["lens"], s["ring"], s["state"])
        s["ws"] = torch.empty(c.paged_tables_workspace_bytes(n), dtype=torch.uint8, device=DEV)
    return s


# ----------------------------------------------------------------------- run


def run(s):
    op = s["case"]["op"]
    if own:
        return {"write": _own_write, "decode": _own_decode, "prefill": _own_prefill, "tables": _own_tables}[op](s)
    return {"write": _plain_write, "decode": _plain_decode, "prefill": _plain_prefill, "tables": _plain_tables}[op](s)


def _own_write(s):
    c, n = s["cache"], s["case"]["n"]
    c.reshape_and_cache(-1, s["k"], s["v"], s["slots"], n)
    c.gather_cached_rows(-1, s["slots"], n, s["k_out"], s["v_out"])
    return {"k": s["k_out"], "v": s["v_out"]}


def _own_decode(s):
    c, hq = s["cache"], s["case"]["H"] * s["case"]["G"]
    if "h_plan" in s:
        c.paged_decode_attention_planned(0, s["q"], hq, s["table"], s["mb"], s["d_plan"], s["h_plan"], s["out"], s["ws"])
    else:
        c.paged_decode_attention(0, s["q"], hq, s["table"], s["mb"], s["lens"], s["n"], s["out"], s["ws"])
    return s["out"]


def _own_prefill(s):
    hq = s["case"]["H"] * s["case"]["G"]
    s["cache"].paged_prefill_attention_staged(0, s["q"], hq, s["table"], s["mb"], s["start"], s["lens"], s["n"], s["out"],
                                              s["ws"], d_sched=s["sched"], n_items=s["n_items"])
    return s["out"]


def _own_tables(s):
    s["cache"].paged_tables_append(s["dt"], s["rows"], s["counts"], s["case"]["n"], s["T"], slots=s["slots"],
                                   positions=s["positions"], chunk_start=s["start"], block_table=s["block_table"],
                                   context_lens=s["context"], lens_out=s["lens_out"], free_state_out=s["state_out"],
                                   workspace=s["ws"])
    return {k: s[k] for k in ("slots", "positions", "start", "block_table", "context", "lens_out", "state_out", "tables")}


def _plain_write(s):
    B, D = s["case"]["B"], s["case"]["D"]
    blk, o = s["slots"] // B, s["slots"] % B
    out = {}
    for name in ("k", "v"):
        codes, scales = _parts(s[name + "_pool"], B, D, name)
        q, d = _quantize(s[name].float().unflatten(-1, (D // 32, 32)))  # [L, n, H, D/32, 32], [L, n, H, D/32]
        codes[:, blk, :, :, o] = _nibbles(q).transpose(0, 1)
        scales[:, blk, :, o] = d.transpose(0, 1)
        x = _values(codes[:, blk, :, :, o], scales[:, blk, :, o])  # [n, L, H, D/32, 32]
        out[name] = x.transpose(0, 1).flatten(-2).contiguous()
    return out


def _rows(s, name):
    """The listed sequences' rows as float32 [n, H, max_blocks * B, D]."""
    codes, scales = _parts(s[name + "_pool"], s["case"]["B"], s["case"]["D"], name)
    at = s["table"].long().clamp(min=0)
    x = _values(codes[0][at], scales[0][at].transpose(-1, -2))  # [n, mb, H, D/32, B, 32]
    return x.permute(0, 2, 1, 4, 3, 5).flatten(4).flatten(2, 3)


def _plain_decode(s):
    c = s["case"]
    H, G, D = c["H"], c["G"], c["D"]
    q = s["q"].float().unflatten(1, (H, G))
    x = torch.matmul(q, _rows(s, "k").transpose(-1, -2)) / math.sqrt(D)
    past = torch.arange(x.shape[-1], device=DEV) >= s["lens"][:, None, None, None]
    x = x.masked_fill(past, -math.inf)
    p = torch.exp(x - x.amax(-1, keepdim=True))
    o = torch.matmul(p, _rows(s, "v")) / p.sum(-1, keepdim=True)
    return o.flatten(1, 2).bfloat16()


def _plain_prefill(s):
    c = s["case"]
    H, G, D, C = c["H"], c["G"], c["D"], s["max_chunk"]
    start, lens = s["start"].long(), s["lens"].long()
    cnt = start[1:] - start[:-1]
    i = torch.arange(C, device=DEV)
    row = (start[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"].float()[row].unflatten(2, (H, G)).permute(0, 2, 3, 1, 4).flatten(2, 3)  # [n, H, G * C, D]
    x = torch.matmul(q, _rows(s, "k").transpose(-1, -2)) / math.sqrt(D)
    pos = (lens - cnt)[:, None] + i  # [n, C]
    past = torch.arange(x.shape[-1], device=DEV) > pos[:, None, None, :, None]
    x = x.unflatten(2, (G, C)).masked_fill(past, -math.inf).flatten(2, 3)
    p = torch.exp(x - x.amax(-1, keepdim=True))
    o = torch.matmul(p, _rows(s, "v")) / p.sum(-1, keepdim=True)
    o = o.unflatten(2, (G, C)).permute(0, 3, 1, 2, 4).flatten(2, 3)  # [n, C, Hq, D]
    t = torch.arange(s["q"].shape[0], device=DEV)
    seq = torch.searchsorted(start[1:], t, right=True)
    return o[seq, t - start[seq]].bfloat16()


def _plain_tables(s):
    B, R, n, mb = (s["case"][x] for x in ("B", "rows", "n", "mb"))
    rows, cnt, T, cap = s["rows"].long(), s["counts"].long(), s["T"], s["ring"].numel()
    old = s["lens"][rows].long()
    new = old + cnt
    ob, nb = (old + B - 1) // B, (new + B - 1) // B
    need = nb - ob
    first = s["state"][0] + torch.cumsum(need, 0) - need
    start = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), torch.cumsum(cnt, 0)])
    j = torch.arange(mb, device=DEV)
    was = s["tables"][rows].long()
    fresh = s["ring"].long()[(first[:, None] + j - ob[:, None]) % cap]
    table = torch.where(j < ob[:, None], was, torch.where(j < nb[:, None], fresh, -1))
    t = torch.arange(T, device=DEV)
    seq = torch.searchsorted(start[1:], t, right=True).clamp(max=n - 1)
    pos = old[seq] + t - start[seq]
    real = t < start[-1]
    slot = table[seq, (pos // B).clamp(max=mb - 1)] * B + pos % B
    s["tables"][rows] = table.int()
    lens_out = s["lens"].clone()
    lens_out[rows] = new.int()
    taken = need.sum()
    return {"slots": torch.where(real, slot, -1), "positions": torch.where(real, pos, -1).int(), "start": start.int(),
            "block_table": table.int(), "context": new.int(), "lens_out": lens_out,
            "state_out": torch.stack([(s["state"][0] + taken) % cap, s["state"][1] - taken]), "tables": s["tables"]}


# ---------------------------------------------------------------------- work


def work(case):
    op = case["op"]
    if op == "write":
        e = 2 * case["L"] * case["n"] * case["H"] * case["D"]  # K and V values
        return {"bytes": e * (2 + 18 / 32 * 2 + 4) + 2 * 8 * case["n"], "flops": 4 * e}
    if op == "decode":
        H, G, D, B = case["H"], case["G"], case["D"], case["B"]
        lens = _lens(case)
        if case["n_br"] > 1:
            toks = sum(int(c) // B * B + case["n_br"] * (int(c) % B + 1) for c in lens)
            ctx, n = sum(case["n_br"] * (int(c) + 1) for c in lens), len(lens) * case["n_br"]
        else:
            toks, ctx, n = int(lens.sum()), int(lens.sum()), len(lens)
        return {"bytes": toks * H * 2 * D * 18 / 32 + n * H * G * D * 4, "flops": 4.0 * D * H * G * ctx}
    if op == "prefill":
        H, G, D = case["H"], case["G"], case["D"]
        hist, chunk = _ints(case["hist"]), _ints(case["chunk"])
        pairs = sum(c * h + c * (c + 1) // 2 for h, c in zip(hist, chunk))
        return {"bytes": sum(hist + chunk) * H * 2 * D * 18 / 32 + sum(chunk) * H * G * D * 4,
                "flops": 4.0 * D * H * G * pairs}
    old, cnt = _counts(case)
    B, n, T = case["B"], case["n"], int(cnt.sum()) + 5
    held, end = -(-old.astype(np.int64) // B), -(-(old.astype(np.int64) + cnt) // B)
    # read: the rows' ids, the ring's, rows, counts, lengths; written: new ids in the rows, the compact table,
    # slots, positions, starts, contexts, lengths
    nbytes = 4 * int(held.sum()) + 8 * int((end - held).sum()) + 4 * n * case["mb"] + 12 * T + 20 * n + 8 * case["rows"]
    return {"bytes": nbytes, "flops": 0}


# --------------------------------------------------------------------- exact


def exact(case, seed):
    """Outputs in 64 bits, one sequence and head (or one token) at a time."""
    if case["op"] == "tables":
        return None  # whole numbers
    s = _inputs(case, seed)
    return {"write": _exact_write, "decode": _exact_decode, "prefill": _exact_prefill}[case["op"]](s)


def _inputs(case, seed):
    global own
    was, own = own, False
    try:
        return prepare(case, seed)
    finally:
        own = was


def _exact_write(s):
    out = {}
    for name in ("k", "v"):
        x = s[name].double()
        g = x.reshape(*x.shape[:-1], -1, 32)
        top = torch.max(g, -1, keepdim=True).values.maximum(-torch.min(g, -1, keepdim=True).values)
        d = (top.float() / 7.0).to(torch.float16).double()  # the scale as the format stores it
        # x / d is rounded to float32 by the format before it goes to the nearest code
        code = torch.nan_to_num((g.float() / d.float()), nan=0.0, posinf=0.0, neginf=0.0).double().round()
        out[name] = (code.clip(-7.0, 7.0) * d).reshape(x.shape)
    return out


def _exact_rows(s, name, ids, h, length, B, D):
    """float64 [length, D] of one sequence and head, through the chunk's bytes."""
    chunk = s[name + "_pool"][0, ids.long(), h]  # [nb, bytes]
    code = chunk[:, : B * D // 2].reshape(-1, D // 32, B, 16).permute(0, 2, 1, 3)  # [nb, B, D/32, 16]
    d = chunk[:, B * D // 2 :].contiguous().view(torch.float16).double()
    d = d.reshape(-1, B, D // 32) if name == "k" else d.reshape(-1, D // 32, B).permute(0, 2, 1)
    lo, hi = (code % 16).double() - 8.0, (code // 16).double() - 8.0
    x = torch.empty(*code.shape[:3], 32, dtype=torch.float64, device=DEV)
    x[..., 0::2], x[..., 1::2] = lo * d[..., None], hi * d[..., None]
    return x.reshape(-1, D)[:length]


def _exact_decode(s):
    c = s["case"]
    B, H, G, D = c["B"], c["H"], c["G"], c["D"]
    out = torch.zeros(s["n"], H * G, D, dtype=torch.float64, device=DEV)
    for i, length in enumerate(s["lens"].tolist()):
        ids = s["table"][i, : -(-length // B)]
        for h in range(H):
            K, V = (_exact_rows(s, x, ids, h, length, B, D) for x in "kv")
            w = torch.softmax(s["q"][i, h * G : (h + 1) * G].double() @ K.T * D**-0.5, -1)
            out[i, h * G : (h + 1) * G] = w @ V
    return out


def _exact_prefill(s):
    c = s["case"]
    B, H, G, D = c["B"], c["H"], c["G"], c["D"]
    hist, chunk = _ints(c["hist"]), _ints(c["chunk"])
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    at = 0
    for i, (past, n) in enumerate(zip(hist, chunk)):
        ids = s["table"][i, : -(-(past + n) // B)]
        seen = torch.ones(n, past + n, dtype=torch.bool, device=DEV).tril(past)
        for h in range(H):
            K, V = (_exact_rows(s, x, ids, h, past + n, B, D) for x in "kv")
            for e in range(h * G, (h + 1) * G):
                x = s["q"][at : at + n, e].double() @ K.T * D**-0.5
                out[at : at + n, e] = torch.softmax(torch.where(seen, x, float("-inf")), -1) @ V
        at += n
    return out
