"""Block tables built on the device against a host model written from the
block manager's rules (new blocks from the front of a FIFO when a token lands
past a row's last block, in batch order; released blocks to its end), alone,
refused, captured into a graph, and driving a q4_0 pool's prefill and decode."""

import collections

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

I32 = dict(dtype=torch.int32, device="cuda")


class Model:
    def __init__(self, n_rows, max_blocks, B, free):
        self.rows = [[] for _ in range(n_rows)]
        self.lens = [0] * n_rows
        self.mb, self.B, self.free = max_blocks, B, collections.deque(free)

    def append(self, rows, counts):
        slots, pos, start = [], [], [0]
        for r, c in zip(rows, counts):
            for _ in range(c if r >= 0 else 0):
                t = self.lens[r]
                if t // self.B == len(self.rows[r]):
                    self.rows[r].append(self.free.popleft())
                slots.append(self.rows[r][t // self.B] * self.B + t % self.B)
                pos.append(t)
                self.lens[r] += 1
            start.append(len(slots))
        return slots, pos, start

    def release(self, rows):
        for r in rows:
            if r >= 0:
                self.free.extend(self.rows[r])
                self.rows[r], self.lens[r] = [], 0


class Device:
    """Table set, outputs and workspace of one test."""

    def __init__(self, n_rows, max_blocks, B, free, cap=None, N=None, head=0):
        from paged_kv_cache_65_gb300 import DeviceTables, PagedKVCache

        cap = cap or len(free)
        N = N or max(free) + 1
        self.c = PagedKVCache(1, N, B, 1, 64, "bf16")
        ring = np.full(cap, -9, dtype=np.int32)
        ring[(head + np.arange(len(free))) % cap] = free
        self.t = DeviceTables(torch.full((n_rows, max_blocks), -1, **I32),
                              torch.zeros(n_rows, **I32), torch.from_numpy(ring).cuda(),
                              torch.tensor([head, len(free)], dtype=torch.int64, device="cuda"))

    def append(self, rows, counts, max_tokens, **kw):
        n = len(counts) if counts is not None else len(rows)
        R, mb = self.t.tables.shape
        out = dict(slots=torch.full((max_tokens,), 77, dtype=torch.int64, device="cuda"),
                   positions=torch.full((max_tokens,), 77, **I32),
                   chunk_start=torch.full((n + 1,), 77, **I32),
                   block_table=torch.full((n, mb), 77, **I32),
                   context_lens=torch.full((n,), 77, **I32))
        ws = torch.empty(self.c.paged_tables_workspace_bytes(n), dtype=torch.uint8, device="cuda")
        d_rows = None if rows is None else torch.tensor(rows, **I32)
        d_counts = None if counts is None else torch.tensor(counts, **I32)
        self.c.paged_tables_append(self.t, d_rows, d_counts, n, max_tokens, workspace=ws, **out, **kw)
        return {k: v.cpu().numpy() for k, v in out.items()}

    def release(self, rows):
        ws = torch.empty(self.c.paged_tables_workspace_bytes(len(rows)), dtype=torch.uint8,
                         device="cuda")
        self.c.paged_tables_release(self.t, torch.tensor(rows, **I32), len(rows), ws)

    def ring(self):
        head, count = self.t.free_state.tolist()
        ids = self.t.free_ids.cpu().numpy()
        return ids[(head + np.arange(count)) % len(ids)].tolist()

    def same(self, m):
        tables = self.t.tables.cpu().numpy()
        want = np.full_like(tables, -1)
        for r, row in enumerate(m.rows):
            want[r, :len(row)] = row
        assert np.array_equal(tables, want)
        assert self.t.lens.cpu().tolist() == m.lens
        assert self.ring() == list(m.free)


def check_append(d, m, rows, counts, max_tokens, **kw):
    got = d.append(rows, counts, max_tokens, **kw)
    full = list(range(len(counts))) if rows is None else rows
    cnt = [1] * len(full) if counts is None else counts
    slots, pos, start = m.append(full, cnt)
    pad = [-1] * (max_tokens - len(slots))
    assert got["slots"].tolist() == slots + pad
    assert got["positions"].tolist() == pos + pad
    assert got["chunk_start"].tolist() == start
    for i, r in enumerate(full):
        row = m.rows[r] if r >= 0 else []
        assert got["block_table"][i].tolist() == row + [-1] * (m.mb - len(row))
        assert got["context_lens"][i] == (m.lens[r] if r >= 0 else 0)
    return got


@pytest.mark.parametrize("seed,n_rows,mb,B", [(0, 7, 5, 16), (1, 40, 9, 8), (2, 3, 300, 1), (3, 1500, 4, 32),
                                              (4, 9, 2100, 16), (5, 64, 33, 7)])
def test_random_appends_and_releases(seed, n_rows, mb, B):
    rng = np.random.default_rng(seed)
    n_free = min(n_rows * mb, 6000)
    free = rng.permutation(n_free + 50)[:n_free].astype(np.int32)
    d = Device(n_rows, mb, B, free, cap=n_free + int(rng.integers(0, 40)), N=n_free + 50,
               head=int(rng.integers(0, n_free)))
    m = Model(n_rows, mb, B, free.tolist())
    for _ in range(12):
        n = int(rng.integers(1, n_rows + 1))
        rows = rng.permutation(n_rows)[:n]
        room = np.array([mb * B - m.lens[r] for r in rows])
        budget = len(m.free) // n
        counts = np.minimum(room, rng.integers(0, max(2, min(3 * B, budget * B)), n))
        need = sum(-(-(m.lens[r] + c) // B) - len(m.rows[r]) for r, c in zip(rows, counts))
        if need > len(m.free):
            counts[:] = 0
        pad = int(rng.integers(0, 3))  # padding entries anywhere in the batch
        at = sorted(rng.integers(0, n + 1, pad))
        rows, counts = list(rows), list(counts)
        for k in at[::-1]:
            rows.insert(k, -1)
            counts.insert(k, int(rng.integers(0, 9)))
        rows, counts = [int(r) for r in rows], [int(c) for c in counts]
        total = sum(c for r, c in zip(rows, counts) if r >= 0)
        check_append(d, m, rows, counts, total + int(rng.integers(0, 3)) * 11)
        d.same(m)
        gone = [int(r) for r in rng.permutation(n_rows)[:int(rng.integers(0, n_rows // 2 + 1))]]
        if gone:
            gone.insert(1, -1)
            d.release(gone)
            m.release(gone)
            d.same(m)
    assert d.c.kv_pool_device_status() == 0


def test_defaults_are_one_token_for_every_row():
    d = Device(5, 3, 4, [9, 3, 7, 1, 0, 5, 2])
    m = Model(5, 3, 4, [9, 3, 7, 1, 0, 5, 2])
    for _ in range(4):
        ws = torch.empty(d.c.paged_tables_workspace_bytes(5), dtype=torch.uint8, device="cuda")
        slots = torch.empty(5, dtype=torch.int64, device="cuda")
        d.c.paged_tables_append(d.t, None, None, 5, 5, slots=slots, workspace=ws)
        assert slots.tolist() == m.append(range(5), [1] * 5)[0]
        d.same(m)


def test_state_written_elsewhere_leaves_the_input_state():
    free = list(range(20, 0, -1))
    d, m = Device(4, 6, 8, free), Model(4, 6, 8, free)
    check_append(d, m, [2, 0], [13, 8], 21)
    lens0, state0 = d.t.lens.clone(), d.t.free_state.clone()
    lens1, state1 = torch.full((4,), 5, **I32), torch.zeros(2, dtype=torch.int64, device="cuda")
    first = d.append([2, 1, 0], [9, 1, 1], 16, lens_out=lens1, free_state_out=state1)
    assert torch.equal(d.t.lens, lens0) and torch.equal(d.t.free_state, state0)
    again = d.append([2, 1, 0], [9, 1, 1], 16, lens_out=lens1, free_state_out=state1)
    assert all(np.array_equal(first[k], again[k]) for k in first)
    slots, _, _ = m.append([2, 1, 0], [9, 1, 1])
    assert first["slots"].tolist() == slots + [-1] * 5
    assert lens1.tolist() == m.lens
    assert state1[1].item() == len(m.free) and int(state1[0]) == (int(state0[0]) + 3) % 20
    d.t.lens.copy_(lens1)
    d.t.free_state.copy_(state1)
    d.same(m)


@pytest.mark.parametrize("rows,counts,max_tokens,bit", [
    ([0, 0], [1, 1], 8, "row"), ([0, 5], [1, 1], 8, "row"), ([-2, 1], [1, 1], 8, "row"),
    ([0, 1], [1, -1], 8, "row"), ([0, 1], [33, 1], 64, "row"), ([0, 1], [2**31 - 1, 1], 64, "row"),
    ([2, 1], [1, 1], 8, "row"), ([3, 1], [1, 1], 8, "row"), ([0, 1], [5, 4], 8, "row"),
    ([0, 1], [32, 9], 64, "free"), ([0, 1, -1], [16, 25, 3], 64, "free")])
def test_refused_batches_change_nothing(rows, counts, max_tokens, bit):
    # rows of up to 4 blocks of 8 tokens; 5 free blocks; row 2 holds a length
    # past its room and row 3 a negative one
    from paged_kv_cache_65_gb300 import _lib

    d = Device(5, 4, 8, [3, 1, 4, 0, 2], cap=9, head=6)
    d.t.lens[2], d.t.lens[3] = 33, -1
    before = [x.clone() for x in (d.t.tables, d.t.lens, d.t.free_ids, d.t.free_state)]
    got = d.append(rows, counts, max_tokens)
    assert d.c.kv_pool_device_status() == (
        _lib.KV_DEV_BAD_TABLE_ROW if bit == "row" else _lib.KV_DEV_NO_FREE_BLOCK)
    for x, y in zip(before, (d.t.tables, d.t.lens, d.t.free_ids, d.t.free_state)):
        assert torch.equal(x, y)
    assert (got["slots"] == -1).all() and (got["positions"] == -1).all()
    assert (got["chunk_start"] == 0).all() and (got["context_lens"] == 0).all()
    assert (got["block_table"] == -1).all()


@pytest.mark.parametrize("state", [[-1, 3], [9, 3], [0, -1], [0, 10]])
def test_a_broken_ring_is_refused(state):
    from paged_kv_cache_65_gb300 import _lib

    d = Device(5, 4, 8, [3, 1, 4, 0, 2], cap=9)
    d.t.free_state.copy_(torch.tensor(state))
    d.append([0], [9], 9)
    assert d.c.kv_pool_device_status() == _lib.KV_DEV_BAD_TABLE_ROW
    d.release([1])
    assert d.c.kv_pool_device_status() == _lib.KV_DEV_BAD_TABLE_ROW
    assert d.t.free_state.tolist() == state and int(d.t.lens.sum()) == 0


def test_release_refuses_repeated_rows_and_a_full_ring():
    from paged_kv_cache_65_gb300 import _lib

    d, m = Device(4, 4, 8, [3, 1, 4, 0, 2]), Model(4, 4, 8, [3, 1, 4, 0, 2])
    check_append(d, m, [1, 3], [9, 8], 17)
    for rows in ([1, 1], [4], [-2, 1]):
        d.release(rows)
        assert d.c.kv_pool_device_status() == _lib.KV_DEV_BAD_TABLE_ROW
        d.same(m)
    d.t.free_state[1] = 4  # 4 free of 5: no room for two blocks
    d.release([1])
    assert d.c.kv_pool_device_status() == _lib.KV_DEV_BAD_TABLE_ROW
    d.t.free_state[1] = 2
    d.release([3, 1])
    m.release([3, 1])
    d.same(m)


def test_ring_ids_outside_the_pool_are_flagged():
    from paged_kv_cache_65_gb300 import _lib

    d = Device(2, 4, 8, [1, 50, 2], N=6)
    got = d.append([0], [20], 20)
    assert d.c.kv_pool_device_status() == _lib.KV_DEV_BAD_BLOCK_ID
    assert got["slots"].tolist() == list(range(8, 16)) + [-1] * 8 + list(range(16, 20))


def test_argument_checks():
    from paged_kv_cache_65_gb300 import DeviceTables, KVError, PagedKVCache, _lib

    d = Device(4, 4, 8, [0, 1, 2])
    ws = torch.empty(d.c.paged_tables_workspace_bytes(4), dtype=torch.uint8, device="cuda")
    rows = torch.zeros(1, **I32)

    def status(call):
        with pytest.raises(KVError) as e:
            call()
        return e.value.status

    bad = _lib.KV_ERR_INVALID_ARG
    assert status(lambda: d.c.paged_tables_append(d.t, rows, None, 1, -1, workspace=ws)) == bad
    assert status(lambda: d.c.paged_tables_append(d.t, rows, None, -1, 1, workspace=ws)) == bad
    assert status(lambda: d.c.paged_tables_append(d.t, None, None, 5, 5, workspace=ws)) == bad
    assert status(lambda: d.c.paged_tables_append(d.t, rows, None, 1, 1, workspace=None)) == bad
    assert status(lambda: d.c.paged_tables_append(d.t, rows, None, 1, 1, workspace=ws[:16])) == bad
    assert status(lambda: d.c.paged_tables_append(d.t, rows, None, 1, 1, block_table=d.t.tables,
                                                  workspace=ws)) == bad
    assert status(lambda: d.c.paged_tables_release(d.t, rows, 1, None)) == bad
    d.c.paged_tables_append(d.t, rows, None, 0, 0)  # an empty batch
    host = PagedKVCache(1, 8, 8, 1, 64, "bf16", allocate=False)
    assert status(lambda: host.paged_tables_append(d.t, rows, None, 1, 1, workspace=ws)) == bad
    with pytest.raises(TypeError):
        DeviceTables(d.t.tables.long(), d.t.lens, d.t.free_ids, d.t.free_state)
    with pytest.raises(ValueError):
        DeviceTables(d.t.tables, d.t.lens[:2], d.t.free_ids, d.t.free_state)


# ---------------------------------------------- a run of the operators together


def bf16_bits(t):
    return t.view(torch.int16).cpu().numpy().view(np.uint16)


@pytest.mark.parametrize("dtype", ["q4_0", "bf16"])
def test_prefill_decode_release_loop_with_captured_steps(dtype):
    from oracle.attention import decode_attention
    from oracle.kv_store import KVStore
    from oracle.prefill import prefill_attention
    from paged_kv_cache_65_gb300 import PagedKVCache
    from paged_kv_cache_65_gb300.driver import TableRun

    L, N, B, H, G, D, R, mb, nb = 2, 80, 16, 2, 4, 128, 6, 12, 60
    perm = np.random.default_rng(4).permutation(N).astype(np.int32)
    c = PagedKVCache(L, N, B, H, D, dtype, free_order=perm)
    c.k.fill_(0)
    c.v.fill_(0)
    run = TableRun(c, H * G, R, mb, nb, 4, max_tokens=160)
    m = Model(R, mb, B, perm[:nb].tolist())
    st = KVStore(L, N, B, H, D, dtype)
    g = torch.Generator(device="cuda")
    g.manual_seed(8)
    tol = 0.02  # checked tightly by the operators' own tests; here the loop is

    def rand(*shape):
        return torch.randn(*shape, device="cuda", generator=g).bfloat16()

    def write(rows, counts, k, v):
        slots, _, _ = m.append(rows, counts)
        for ly in range(L):
            st.reshape_and_cache(ly, bf16_bits(k[ly]), bf16_bits(v[ly]), slots)

    def context(ly, r):
        return st.gather(ly, m.rows[r], m.lens[r])

    def prefill(rows, counts):
        T = 160
        q, k, v = rand(L, T, H * G, D), rand(L, T, H, D), rand(L, T, H, D)
        out = torch.zeros((L, T, H * G, D), device="cuda")
        run.prefill(torch.tensor(rows, **I32), torch.tensor(counts, **I32), max(counts), q, k, v, out)
        write(rows, counts, k, v)
        for ly in range(L):
            at = 0
            for r, n in zip(rows, counts):
                if r < 0:
                    continue
                kk, vv = context(ly, r)
                ref = prefill_attention(q[ly, at:at + n].float().cpu().numpy(), kk, vv)
                assert np.abs(out[ly, at:at + n].cpu().numpy() - ref).max() <= tol
                at += n
            assert bool((out[ly, at:] == 0).all())

    def step_check(rows, q, k, v, out):
        write(rows, [1] * len(rows), k, v)
        for ly in range(L):
            for i, r in enumerate(rows):
                if r < 0:
                    assert bool((out[ly, i] == 0).all())
                    continue
                kk, vv = context(ly, r)
                ref = decode_attention(q[ly, i].float().cpu().numpy(), kk, vv)
                assert np.abs(out[ly, i].cpu().numpy() - ref).max() <= tol

    prefill([3, 0, 5], [61, 16, 80])
    # a decode step captured once and replayed with other rows and values
    n = 4
    d_rows = torch.tensor([3, 0, 5, -1], **I32)
    q, k, v = rand(L, n, H * G, D), rand(L, n, H, D), rand(L, n, H, D)
    out = torch.zeros((L, n, H * G, D), device="cuda")
    run.step(d_rows, q, k, v, out)  # warm-up, a real step
    torch.cuda.synchronize()
    step_check([3, 0, 5, -1], q, k, v, out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run.step(d_rows, q, k, v, out)
    torch.cuda.synchronize()
    for rows in ([0, 3, 5, -1], [5, 0, 3, -1], [0, -1, -1, -1]) * 6:
        d_rows.copy_(torch.tensor(rows))
        q.copy_(rand(L, n, H * G, D))
        k.copy_(rand(L, n, H, D))
        v.copy_(rand(L, n, H, D))
        graph.replay()
        torch.cuda.synchronize()
        step_check(rows, q, k, v, out)
    run.release(torch.tensor([5], **I32))
    m.release([5])
    prefill([1, 3], [100, 33])
    d_rows.copy_(torch.tensor([1, 3, 0, -1]))
    graph.replay()
    torch.cuda.synchronize()
    step_check([1, 3, 0, -1], q, k, v, out)
    assert run.t.lens.cpu().tolist() == m.lens
    assert c.kv_pool_device_status() == 0
    run.close()
    c.kv_pool_check()
    assert c.kv_pool_stats()[1] == 0


def test_a_run_refuses_what_its_buffers_do_not_hold():
    from paged_kv_cache_65_gb300 import PagedKVCache
    from paged_kv_cache_65_gb300.driver import TableRun

    c = PagedKVCache(1, 16, 16, 2, 128, "q4_0")
    run = TableRun(c, 8, 4, 4, 8, 2)
    rows = torch.tensor([0, 1], **I32)
    kv = torch.zeros((1, 2, 2, 128), dtype=torch.bfloat16, device="cuda")
    q = torch.zeros((1, 2, 8, 128), dtype=torch.bfloat16, device="cuda")
    out = torch.zeros((1, 2, 8, 128), device="cuda")
    one = torch.tensor([1, 1], **I32)
    with pytest.raises(ValueError):  # three rows in a run of two
        run.step(torch.tensor([0, 1, 2], **I32), q, kv, kv, out)
    with pytest.raises(ValueError):  # fewer values than rows
        run.step(rows, q, kv[:, :1].contiguous(), kv, out)
    with pytest.raises(ValueError):  # a run without staging
        run.prefill(rows, one, 1, q, kv, kv, out)
    with pytest.raises(TypeError):
        run.step(rows.long(), q, kv, kv, out)
    run.step(rows, q, kv, kv, out)
    assert run.t.lens.cpu().tolist() == [1, 1, 0, 0]
    assert c.kv_pool_device_status() == 0
    run.close()
