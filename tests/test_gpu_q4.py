"""q4_0 pools on the GPU against the oracle ("第 8 章 推理优化" §8.4.2, Fig.
8-23: 32 values share one fp16 scale, one 4-bit code each): the codes and
scales the slot write stores and copy-on-write copies are bit-exact, rows read
back are exact, and decode attention (plain, planned, without a workspace,
captured into a graph, through host buffers) matches attention in 64 bits over
the dequantized values.

Tolerance of attention.  Weights are p = 2^(s - m + e) with the sum l, values
v = c d (|c| <= 7, n = c + 8 <= 15).  The pass rounds p to fp16 (half a step:
2^-11 relative) and p d again to fp16 (the same), multiplies the twice rounded
product by n and the once rounded p by 8 d, in float32; l sums the rounded p.  So
the sum over T
tokens is off by at most
    sum p d (2^-11 |c| + 2^-11 n)  <=  l (2^-11 + 2^-11 15 / 7) max|v|
                                   =  l 2^-10 1.572 max|v|
plus what fp16 loses below its normal range, at most 2^-25 (|c| d + n) a token.
Against l: e is 14 until a scale d of 2 or more shows, so l >= 2^12 and the loss
vanishes; from then on e is 0, l >= 2^-2 (a maximum moves to 2^-2), and T tokens
lose T 2^-23 (max|v| + 15) at most, with d >= 2 somewhere.  The scores come from
products accumulated in float32: |n Q| <= 15 |Q| over 128 terms and the scales'
sum of four, at most 2^-24 per addition of at most 16 * 128 * max|k scale| *
max|q| * scale * log2(e); an error e_s of s moves an output by at most 2 e_s ln 2
max|v|.  exp2's 2^-22 and the float32 sums are inside the first term's slack:
2^-10 (1.572 + 2^-3).  Errors of random values add up as their root, far below.
"""

import numpy as np
import pytest

import synth
from oracle.attention import decode_attention
from oracle.kv_store import KVStore
from oracle.runner import OracleRun

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def attention_tol(q_max, ks_max, v_max, tokens, d, out="f32"):
    scale = 1.4427 / np.sqrt(d)
    e_s = 2.0**-24 * (d + 8) * 16 * ks_max * q_max * scale
    tol = v_max * (2.0**-10 * 1.697 + 2 * e_s * 0.6932)
    if v_max >= 14:  # a scale of 2 or more
        tol += tokens * (v_max + 15) * 2.0**-23
    return tol + (2.0**-8 * v_max if out == "bf16" else 0.0)


def layout(cache):
    """The device pool as the oracle store lays it out: codes [L, N, B, H,
    D/2], scale bits [L, N, B, H, D/32], for K and V."""
    L, N, B, H, D = cache.L, cache.N, cache.B, cache.H, cache.D
    out = []
    for name, t in (("k", cache.k), ("v", cache.v)):
        a = t.cpu().numpy()
        codes = a[..., : B * D // 2].reshape(L, N, H, D // 32, B, 16)
        sc = np.ascontiguousarray(a[..., B * D // 2:]).view(np.uint16)
        if name == "k":
            sc = sc.reshape(L, N, H, B, D // 32).transpose(0, 1, 3, 2, 4)
        else:
            sc = sc.reshape(L, N, H, D // 32, B).transpose(0, 1, 4, 2, 3)
        out.append((codes.transpose(0, 1, 4, 2, 3, 5).reshape(L, N, B, H, D // 2), sc))
    return out


def same_pool(cache, st):
    (kc, ks), (vc, vs) = layout(cache)
    return (np.array_equal(kc, st.K) and np.array_equal(ks, st.Ks)
            and np.array_equal(vc, st.V) and np.array_equal(vs, st.Vs))


MMA, WIDE = 2, 3  # KV_OPT_DECODE_PATH of plans: the pass's narrow form, its wide form


def make(wl, fill=0, path=0):
    from paged_kv_cache_65_gb300 import PagedKVCache, _lib
    from paged_kv_cache_65_gb300.driver import DeviceRun

    cache = PagedKVCache(wl.n_layers, wl.n_blocks, wl.block_size, wl.n_kv_heads, wl.head_dim,
                         wl.dtype, free_order=wl.free_order)
    cache.kv_pool_set_option(_lib.KV_OPT_DECODE_PATH, path)
    cache.k.fill_(fill)
    cache.v.fill_(fill)
    run = DeviceRun(cache, wl.n_q_heads)
    for op in wl.build_ops:
        run.apply(op, wl.append_values)
    return cache, run


def q4_workload(name, G, B, seed, ctxs, H=2, D=128, fork=None, layers=1):
    n_blocks = (sum(-(-c // B) for c in ctxs) + 2 * len(ctxs)
                + (-(-fork // B) + 6 if fork else 0) + 8)
    ops = [("append", s, c - 1, s) for s, c in enumerate(ctxs) if c > 1]
    seqs = list(range(len(ctxs)))
    if fork is not None:  # a prefix of `fork` tokens forked into two, parent alive
        ops += [("append", 100, fork, 99), ("fork", 100, 101), ("fork", 100, 102)]
        seqs += [100, 101, 102]
    return synth.Workload(name, layers, n_blocks, B, H * G, H, D, "q4_0", seed,
                          synth.permutation((seed, 9), n_blocks), ops, seqs)


def step_tol(orc, q, out="f32"):
    """Tolerance of one decode step of an oracle run (values N(0, 1))."""
    st = orc.st
    ks = st.Ks.view(np.float16).astype(np.float64).max()
    vs = st.Vs.view(np.float16).astype(np.float64).max()
    q_max = np.abs((np.asarray(q).astype(np.uint32) << 16).view(np.float32)).max()
    return attention_tol(q_max, ks, 7 * vs, max(orc.bm.lengths.values()), st.D, out)


def max_err(gpu, ref):
    return float(np.max(np.abs(gpu.astype(np.float64) - ref))) if ref.size else 0.0


# ------------------------------------------------------------------ rows


def dev_bf16(x):
    """float32 array -> bfloat16 device tensor and its exact float32 values."""
    t = torch.from_numpy(np.ascontiguousarray(x)).to(torch.bfloat16)
    return t.cuda(), t.float().numpy()


@pytest.mark.parametrize("L,B,H,D,n", [(1, 8, 1, 64, 1), (2, 16, 3, 128, 29), (1, 64, 8, 128, 200),
                                       (3, 256, 2, 64, 77), (1, 8, 1, 32, 5), (1, 24, 2, 96, 9)])
def test_written_rows_are_the_oracles_codes_and_read_back_exactly(L, B, H, D, n):
    from oracle.q4 import q4_decode, q4_encode
    from paged_kv_cache_65_gb300 import KVError, PagedKVCache

    rng = np.random.default_rng(7 * B + D + n)
    N = -(-n // B) + 3
    c = PagedKVCache(L, N, B, H, D, "q4_0")
    c.k.fill_(0xEE)
    c.v.fill_(0xEE)
    k, kf = dev_bf16(rng.standard_normal((L, n, H, D)).astype(np.float32))
    v, vf = dev_bf16(rng.standard_normal((L, n, H, D)).astype(np.float32) * 100)
    slots = rng.permutation(N * B)[:n].astype(np.int64)
    slots[n // 2] = -1 if n > 1 else slots[0]
    d_slots = torch.from_numpy(slots).cuda()
    if D in (32, 96) or B % 8 or (64 % B and B % 64):  # shapes no device pass takes
        with pytest.raises(KVError):
            c.reshape_and_cache(-1, k, v, d_slots, n)
        return
    c.reshape_and_cache(-1, k, v, d_slots, n)
    (kc, ks), (vc, vs) = layout(c)
    live = slots >= 0
    blk, o = slots[live] // B, slots[live] % B
    for codes, sc, x in ((kc, ks, kf), (vc, vs, vf)):
        want, wsc = q4_encode(x[:, live])
        assert np.array_equal(codes[:, blk, o], want)
        assert np.array_equal(sc[:, blk, o], wsc)
    # untouched slots keep their bytes
    rest = np.ones((N, B), bool)
    rest[blk, o] = False
    for codes, sc in ((kc, ks), (vc, vs)):
        assert (codes[:, rest] == 0xEE).all() and (sc[:, rest] == 0xEEEE).all()
    for dt in (torch.float32, torch.bfloat16):
        ko = torch.full((L, n, H, D), 5.0, dtype=dt, device="cuda")
        vo = torch.full((L, n, H, D), 5.0, dtype=dt, device="cuda")
        c.gather_cached_rows(-1, d_slots, n, ko, vo)
        for got, x in ((ko, kf), (vo, vf)):
            want = torch.from_numpy(q4_decode(*q4_encode(x))).to(torch.float32).to(dt)
            want[:, ~live] = 5.0
            assert torch.equal(got.cpu(), want)
    one = torch.zeros((n, H, D), device="cuda")
    two = torch.zeros((n, H, D), device="cuda")
    c.gather_cached_rows(L - 1, d_slots, n, one, two)
    assert torch.equal(one.cpu()[live], torch.from_numpy(
        q4_decode(*q4_encode(kf[L - 1]))).float()[live])
    assert c.kv_pool_device_status() == 0


def test_groups_of_zeros_tiny_huge_and_extreme_values():
    from oracle.q4 import q4_decode, q4_encode
    from paged_kv_cache_65_gb300 import PagedKVCache

    rng = np.random.default_rng(3)
    n, H, D = 12, 2, 128
    x = rng.standard_normal((1, n, H, D)).astype(np.float32)
    scale = np.array([0.0, 1e-38, 1e-9, 1e-7, 3e-7, 1e-4, 1.0, 1e3, 6e4, 1e5, 4.5e5, 1e-6])
    x *= scale[None, :, None, None].astype(np.float32)
    x = np.clip(x, -4.5e5, 4.5e5)  # 4.5e5 / 7 is the largest a finite fp16 scale holds
    x[0, 6, :, :32] = 0.0
    x[0, 7, :, 5] = -x[0, 7].max() * 2   # a negative largest value
    c = PagedKVCache(1, 4, 16, H, D, "q4_0")
    k, kf = dev_bf16(x)
    slots = torch.arange(n, device="cuda")
    c.reshape_and_cache(0, k, k, slots, n)
    ko = torch.empty((n, H, D), device="cuda")
    vo = torch.empty((n, H, D), device="cuda")
    c.gather_cached_rows(0, slots, n, ko, vo)
    want = torch.from_numpy(q4_decode(*q4_encode(kf[0]))).float()
    assert torch.equal(ko.cpu(), want) and torch.equal(vo.cpu(), want)
    (kc, ks), _ = layout(c)
    codes, sc = q4_encode(kf[0])
    assert np.array_equal(kc[0].reshape(-1, H, D // 2)[:n], codes)
    assert np.array_equal(ks[0].reshape(-1, H, D // 32)[:n], sc)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "fp8_e4m3", "q8_0", "q4_0"])
def test_gather_reads_every_pool_dtype(dtype):
    from paged_kv_cache_65_gb300 import PagedKVCache

    rng = np.random.default_rng(11)
    L, N, B, H, D, n = 2, 5, 16, 3, 128, 21
    c = PagedKVCache(L, N, B, H, D, dtype)
    st = KVStore(L, N, B, H, D, dtype, 0.5, 2.0)
    if dtype == "fp8_e4m3":
        c.kv_pool_set_fp8_scales(0.5, 2.0)
    x = synth.storage_values(rng.standard_normal((2, L, n, H, D)).astype(np.float32), dtype)
    slots = rng.permutation(N * B)[:n].astype(np.int64)
    from paged_kv_cache_65_gb300.driver import to_device

    d_slots = torch.from_numpy(slots).cuda()
    c.reshape_and_cache(-1, to_device(x[0], dtype, "cuda"), to_device(x[1], dtype, "cuda"),
                        d_slots, n)
    for ly in range(L):
        st.reshape_and_cache(ly, x[0][ly], x[1][ly], slots)
    for dt in (torch.float32, torch.bfloat16):
        ko = torch.empty((L, n, H, D), dtype=dt, device="cuda")
        vo = torch.empty((L, n, H, D), dtype=dt, device="cuda")
        c.gather_cached_rows(-1, d_slots, n, ko, vo)
        for ly in range(L):
            for i, s in enumerate(slots):
                k, v = st.gather(ly, [s // B], int(s % B) + 1)
                # products of a code and its scale fit float32 (power-of-two FP8 scales)
                assert torch.equal(ko[ly, i].cpu(), torch.from_numpy(k[-1]).float().to(dt))
                assert torch.equal(vo[ly, i].cpu(), torch.from_numpy(v[-1]).float().to(dt))


def test_slots_past_the_pool_are_skipped_and_flagged():
    from paged_kv_cache_65_gb300 import PagedKVCache, _lib

    c = PagedKVCache(1, 4, 16, 2, 128, "q4_0")
    c.k.fill_(0x11)
    c.v.fill_(0x11)
    rows = torch.ones((2, 2, 128), dtype=torch.bfloat16, device="cuda")
    slots = torch.tensor([4 * 16, -7], device="cuda")
    c.reshape_and_cache(0, rows, rows, slots, 2)
    assert c.kv_pool_device_status() == _lib.KV_DEV_BAD_SLOT
    assert bool((c.k == 0x11).all()) and bool((c.v == 0x11).all())
    out = torch.full((2, 2, 128), 3.0, device="cuda")
    c.gather_cached_rows(0, slots, 2, out, out.clone())
    assert c.kv_pool_device_status() == _lib.KV_DEV_BAD_SLOT
    assert bool((out == 3.0).all())


# ---------------------------------------------------------------- decode


@pytest.mark.parametrize("G,B,D,path", [
    (8, 16, 64, MMA), (4, 8, 64, MMA), (8, 256, 64, MMA), (1, 192, 64, MMA), (2, 32, 64, WIDE),
    *[(G, B, 128, path) for path in (MMA, WIDE) for G, B in ((1, 16), (2, 8), (4, 32), (8, 64), (4, 128), (2, 192),
                                                          (8, 256))]])
def test_decode_of_ragged_contexts(G, B, D, path):
    ctxs = [1, 2, B - 1, B, B + 1, 3 * B + 2, 97, 128, 129, 700]
    wl = q4_workload("q4_ragged", G, B, 30 + G + B, ctxs, D=D)
    orc = OracleRun(wl)
    cache, run = make(wl, path=path)
    so, co, q, outs = orc.step(0)
    _, k, v = wl.step_values(0)
    sg, _, og = run.step(wl.decode_seqs, q, k, v)
    assert list(sg) == so
    assert same_pool(cache, orc.st)
    assert max_err(og.cpu().numpy()[0], outs[0]) <= step_tol(orc, q), (G, B, D)
    assert cache.kv_pool_device_status() == 0


@pytest.mark.parametrize("D,G,B,path", [(128, 4, 16, MMA), (64, 8, 16, MMA), (128, 8, 32, MMA), (128, 1, 8, MMA),
                                        (128, 4, 16, WIDE), (128, 8, 32, WIDE), (128, 1, 8, WIDE), (128, 2, 192, WIDE),
                                        (64, 8, 16, WIDE), (64, 4, 8, WIDE), (64, 2, 32, WIDE), (64, 8, 256, WIDE)])
def test_fork_copy_on_write_and_the_planned_pass(D, G, B, path):
    # two steps over two layers: the first copies the shared, partly filled
    # tail of the forks; the shared prefix is read once through the plan
    wl = q4_workload("q4_fork", G, B, 22, [1, 15, 17, 40, 300], fork=203, D=D, layers=2)
    orc = OracleRun(wl)
    cache, run = make(wl, path=path)
    assert same_pool(cache, orc.st)
    from paged_kv_cache_65_gb300.cache import parse_plan
    from paged_kv_cache_65_gb300.driver import to_device

    for step in range(2):
        so, co, q, outs = orc.step(step)
        _, k, v = wl.step_values(step)
        sg, pg, og = run.step(wl.decode_seqs, q, k, v, planned=True)
        assert list(sg) == so and [tuple(p) for p in pg] == co
        assert len(co) == (2 if step == 0 else 0)
        assert same_pool(cache, orc.st)
        tol = step_tol(orc, q)
        for ly in range(2):
            assert max_err(og.cpu().numpy()[ly], outs[ly]) <= tol
        h_plan, _, _ = run.plan(wl.decode_seqs, run.max_blocks(wl.decode_seqs))
        plan = parse_plan(h_plan)
        assert plan["kernel"] == path and (plan["n_shared_segs"] > 0 or B > 128)
        # the same step per sequence, in bfloat16
        d_table, d_lens, mb = run.tables(wl.decode_seqs)
        qd = to_device(q, "bf16", "cuda")
        got = run.attend(1, qd, d_table, mb, d_lens, len(wl.decode_seqs),
                         out_dtype=torch.bfloat16)
        assert max_err(got.float().cpu().numpy(), outs[1]) <= step_tol(orc, q, "bf16")
    assert cache.kv_pool_device_status() == 0


@pytest.mark.parametrize("path", [MMA, WIDE])
@pytest.mark.parametrize("n_br,G,D", [(3, 4, 128), (4, 8, 128), (8, 4, 128), (5, 1, 128), (2, 8, 64), (4, 8, 64)])
def test_wide_shared_segments(n_br, G, D, path):
    # segments of 12 to 32 columns: two and four n-tiles
    B, H, prefix = 16, 2, 1040
    n_blocks = prefix // B + 3 * n_br + 8
    ops = [("append", 100, prefix, 99)] + [("fork", 100, s) for s in range(n_br)]
    ops += [("append", s, 3 * s, s) for s in range(1, n_br)]
    wl = synth.Workload("q4_wide", 1, n_blocks, B, H * G, H, D, "q4_0", 5,
                        synth.permutation((5, n_br), n_blocks), ops, list(range(n_br)))
    orc = OracleRun(wl)
    cache, run = make(wl, path=path)
    so, co, q, outs = orc.step(0)
    _, k, v = wl.step_values(0)
    sg, _, og = run.step(wl.decode_seqs, q, k, v, planned=True)
    assert list(sg) == so
    assert max_err(og.cpu().numpy()[0], outs[0]) <= step_tol(orc, q)
    assert cache.kv_pool_device_status() == 0


@pytest.mark.parametrize("path", [MMA, WIDE])
@pytest.mark.parametrize("planned", [False, True])
def test_unused_slots_of_nan_scales_do_not_leak(planned, path):
    # every byte of the unused slots is 0xFF: codes of 7, scales with NaN bits
    wl = q4_workload("q4_nan", 4, 16, 23, [1, 15, 17, 70, 333], fork=150)
    orc = OracleRun(wl)
    cache, run = make(wl, fill=0xFF, path=path)
    so, co, q, outs = orc.step(0)
    _, k, v = wl.step_values(0)
    _, _, og = run.step(wl.decode_seqs, q, k, v, planned=planned)
    got = og.cpu().numpy()[0]
    assert np.isfinite(got).all()
    tol = attention_tol(5.0, 1.0, 7.0, 400, 128)
    assert max_err(got, outs[0]) <= tol


@pytest.mark.parametrize("path", [MMA, WIDE])
def test_empty_contexts_give_zeros_and_bad_tables_are_flagged(path):
    from paged_kv_cache_65_gb300 import PagedKVCache, _lib

    c = PagedKVCache(1, 8, 16, 2, 128, "q4_0")
    c.kv_pool_set_option(_lib.KV_OPT_DECODE_PATH, path)
    c.k.zero_()
    c.v.zero_()
    q = torch.ones((3, 8, 128), dtype=torch.bfloat16, device="cuda")
    table = torch.tensor([[0, 1], [2, 3], [4, 5]], dtype=torch.int32, device="cuda")
    ws = torch.empty(c.paged_decode_workspace_bytes(3, 8), dtype=torch.uint8, device="cuda")
    out = torch.full((3, 8, 128), 9.0, device="cuda")
    for lens in ([0, 0, 0], [0, 5, 0]):
        d_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        c.paged_decode_attention(0, q, 8, table, 2, d_lens, 3, out, ws)
        assert bool((out == 0).all())
        assert c.kv_pool_device_status() == 0
    bad = torch.tensor([[0, 8], [-1, 3], [4, 5]], dtype=torch.int32, device="cuda")
    d_lens = torch.tensor([20, 3, 0], dtype=torch.int32, device="cuda")
    c.paged_decode_attention(0, q, 8, bad, 2, d_lens, 3, out, ws)
    assert c.kv_pool_device_status() == _lib.KV_DEV_BAD_BLOCK_ID
    d_lens = torch.tensor([-3, 33, 0], dtype=torch.int32, device="cuda")
    c.paged_decode_attention(0, q, 8, table, 2, d_lens, 3, out, ws)
    assert c.kv_pool_device_status() == _lib.KV_DEV_BAD_CONTEXT


@pytest.mark.parametrize("path", [MMA, WIDE])
@pytest.mark.parametrize("q_scale,k_scale,v_scale", [(1e-3, 1.0, 1.0), (30.0, 1.0, 1.0), (1.0, 1e-4, 1e-3),
                                                     (1e5, 1e-4, 1.0), (1e-6, 5e4, 4e4), (1.0, 8.0, 5e4)])
def test_magnitudes_of_q_k_and_v(q_scale, k_scale, v_scale, path):
    from paged_kv_cache_65_gb300 import PagedKVCache, _lib

    rng = np.random.default_rng(41)
    n, B, H, G, D = 300, 16, 2, 4, 128
    c = PagedKVCache(1, 20, B, H, D, "q4_0")
    c.kv_pool_set_option(_lib.KV_OPT_DECODE_PATH, path)
    st = KVStore(1, 20, B, H, D, "q4_0")
    xk = synth.storage_values((rng.standard_normal((n, H, D)) * k_scale).astype(np.float32), "q4_0")
    xv = synth.storage_values((rng.standard_normal((n, H, D)) * v_scale).astype(np.float32), "q4_0")
    slots = np.arange(n, dtype=np.int64)
    to = lambda x: torch.from_numpy(x.view(np.int16)).cuda().view(torch.bfloat16)  # noqa: E731
    c.reshape_and_cache(0, to(xk), to(xv), torch.from_numpy(slots).cuda(), n)
    st.reshape_and_cache(0, xk, xv, slots)
    q, qf = dev_bf16(rng.standard_normal((1, H * G, D)).astype(np.float32) * q_scale)
    table = torch.arange(20, dtype=torch.int32, device="cuda").reshape(1, 20)
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    ws = torch.empty(c.paged_decode_workspace_bytes(1, H * G), dtype=torch.uint8, device="cuda")
    out = torch.empty((1, H * G, D), device="cuda")
    c.paged_decode_attention(0, q, H * G, table, 20, lens, 1, out, ws)
    k, v = st.gather(0, list(range(20)), n)
    ref = decode_attention(qf[0], k, v)
    tol = attention_tol(np.abs(qf).max(), np.abs(st.Ks.view(np.float16)).max().astype(np.float64),
                        np.abs(v).max(), n, D)
    assert max_err(out.cpu().numpy()[0], ref) <= tol


@pytest.mark.parametrize("path,D,B", [(MMA, 128, 16), (WIDE, 128, 8), (WIDE, 64, 192), (MMA, 64, 64), (WIDE, 128, 256)])
@pytest.mark.parametrize("low,high,at", [(1e-5, 100.0, 700), (1e-3, 20.0, 33), (60.0, 1e-4, 500), (1e-6, 1e-6, 0)])
def test_v_scales_that_grow_and_shrink_along_a_sequence(low, high, at, path, D, B):
    # values of the first `at` tokens around `low`, then around `high`, the
    # groups a factor of 4 apart: the weights' range moves inside the sequence
    from paged_kv_cache_65_gb300 import PagedKVCache, _lib

    rng = np.random.default_rng(43)
    n, H, G, n_br = 1100, 2, 8, 3
    nb = -(-n // B)
    c = PagedKVCache(1, nb + 4, B, H, D, "q4_0")
    c.kv_pool_set_option(_lib.KV_OPT_DECODE_PATH, path)
    st = KVStore(1, nb + 4, B, H, D, "q4_0")
    slots, pairs = c.seq_append_tokens(0, n)
    scale = np.where(np.arange(n) < at, low, high)[:, None, None] * 0.25 ** (np.arange(D) // 32)
    xk = synth.storage_values(rng.standard_normal((n, H, D)).astype(np.float32), "q4_0")
    xv = synth.storage_values((rng.standard_normal((n, H, D)) * scale).astype(np.float32), "q4_0")
    to = lambda x: torch.from_numpy(x.view(np.int16)).cuda().view(torch.bfloat16)  # noqa: E731
    c.reshape_and_cache(0, to(xk), to(xv), torch.from_numpy(np.asarray(slots)).cuda(), n)
    st.reshape_and_cache(0, xk, xv, slots)
    for s in (1, 2):
        c.seq_fork(0, s)
    q, qf = dev_bf16(rng.standard_normal((n_br, H * G, D)).astype(np.float32))
    table, _ = c.seq_block_table(list(range(n_br)), nb)
    h_plan, ws_bytes = c.paged_decode_plan(list(range(n_br)), H * G, nb)
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device="cuda")
    out = torch.empty((n_br, H * G, D), device="cuda")
    d_table = torch.from_numpy(np.ascontiguousarray(table)).cuda()
    c.paged_decode_attention_planned(0, q, H * G, d_table, nb, torch.from_numpy(h_plan).cuda(), h_plan, out, ws)
    k, v = st.gather(0, list(table[0]), n)
    ks = st.Ks.view(np.float16).astype(np.float64).max()
    for i in range(n_br):
        ref = decode_attention(qf[i], k, v)
        got = out[i].cpu().numpy()
        for g in range(D // 32):  # each group against its own values
            d = slice(32 * g, 32 * g + 32)
            v_max = np.abs(v[..., d]).max()
            tol = attention_tol(np.abs(qf).max(), ks, v_max, n, D)
            if np.abs(v).max() >= 14 and v_max < 14:
                tol += n * (v_max + 15) * 2.0**-23
            assert max_err(got[:, d], ref[:, d]) <= tol, (i, g)
    assert c.kv_pool_device_status() == 0


@pytest.mark.parametrize("planned,path", [(False, MMA), (True, MMA), (True, WIDE)])
@pytest.mark.parametrize("G,B,D", [(8, 8, 128), (4, 16, 64), (1, 64, 128)])
def test_few_long_segments_of_one_head(G, B, D, planned, path):
    # less work than teams over long segments: the split takes its least chunk,
    # and short sequences share chunks with the long ones
    wl = q4_workload("q4_least", G, B, 47, [9001, 3, 2500, 64], H=1, D=D, fork=6007)
    orc = OracleRun(wl)
    cache, run = make(wl, path=path)
    for step in range(2):  # the second plan's start records know the launch
        so, co, q, outs = orc.step(step)
        _, k, v = wl.step_values(step)
        sg, _, og = run.step(wl.decode_seqs, q, k, v, planned=planned)
        assert list(sg) == so
        assert max_err(og.cpu().numpy()[0], outs[0]) <= step_tol(orc, q)
    assert cache.kv_pool_device_status() == 0


@pytest.mark.parametrize("path", [MMA, WIDE])
def test_long_context_and_offsets_past_32_bits(path):
    # a pool whose byte offsets pass 2^32 and one sequence through its last blocks
    from paged_kv_cache_65_gb300 import PagedKVCache, _lib

    B, H, D, G, N = 32, 8, 128, 8, 260000  # N * H * B * 72 bytes = 4.8e9 of K
    c = PagedKVCache(1, N, B, H, D, "q4_0")
    c.kv_pool_set_option(_lib.KV_OPT_DECODE_PATH, path)
    n = 5000
    rng = np.random.default_rng(2)
    nb = -(-n // B)
    blocks = np.concatenate([np.arange(N - nb + 3, N), [0, 7, N // 2]])[:nb].astype(np.int32)
    rng.shuffle(blocks)
    t = np.arange(n)
    slots = blocks[t // B].astype(np.int64) * B + t % B
    k, kf = dev_bf16(rng.standard_normal((n, H, D)).astype(np.float32))
    v, vf = dev_bf16(rng.standard_normal((n, H, D)).astype(np.float32))
    d_slots = torch.from_numpy(slots).cuda()
    c.reshape_and_cache(0, k, v, d_slots, n)
    from oracle.q4 import q4_decode, q4_encode

    ref_k, ref_v = q4_decode(*q4_encode(kf)), q4_decode(*q4_encode(vf))
    ko = torch.empty((n, H, D), device="cuda")
    vo = torch.empty((n, H, D), device="cuda")
    c.gather_cached_rows(0, d_slots, n, ko, vo)
    assert np.array_equal(ko.cpu().numpy(), ref_k.astype(np.float32))
    assert np.array_equal(vo.cpu().numpy(), ref_v.astype(np.float32))
    q, qf = dev_bf16(rng.standard_normal((1, H * G, D)).astype(np.float32))
    table = torch.from_numpy(blocks).reshape(1, nb).cuda()
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    ws = torch.empty(c.paged_decode_workspace_bytes(1, H * G), dtype=torch.uint8, device="cuda")
    out = torch.empty((1, H * G, D), device="cuda")
    c.paged_decode_attention(0, q, H * G, table, nb, lens, 1, out, ws)
    ref = decode_attention(qf[0], ref_k, ref_v)
    tol = attention_tol(np.abs(qf).max(), 1.0, np.abs(ref_v).max(), n, D)
    assert max_err(out.cpu().numpy()[0], ref) <= tol
    assert c.kv_pool_device_status() == 0


@pytest.mark.parametrize("path", [MMA, WIDE])
def test_without_a_workspace_on_another_stream_and_in_a_graph(path):
    wl = q4_workload("q4_graph", 4, 16, 61, [5, 64, 333, 1000])
    orc = OracleRun(wl)
    cache, run = make(wl, path=path)
    so, co, q, outs = orc.step(0)
    _, k, v = wl.step_values(0)
    sg, _, og = run.step(wl.decode_seqs, q, k, v)
    ref = og[0].clone()
    assert max_err(ref.cpu().numpy(), outs[0]) <= step_tol(orc, q)
    from paged_kv_cache_65_gb300.driver import to_device

    n, hq = len(wl.decode_seqs), wl.n_q_heads
    qd = to_device(q, "bf16", "cuda")
    d_table, d_lens, mb = run.tables(wl.decode_seqs)
    out = torch.empty_like(ref)
    cache.paged_decode_attention_noalloc(0, qd, hq, d_table, mb, d_lens, n, out)
    assert torch.equal(out, ref)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    out2 = torch.zeros_like(ref)
    ws = torch.empty(cache.paged_decode_workspace_bytes(n, hq), dtype=torch.uint8, device="cuda")
    cache.paged_decode_attention(0, qd, hq, d_table, mb, d_lens, n, out2, ws, stream=side)
    side.synchronize()
    assert torch.equal(out2, ref)
    # a captured step: slot write of a row, read-back, attention
    rows = torch.randn((1, 2, 128), device="cuda").bfloat16()
    slot = torch.tensor([int(sg[0])], device="cuda")
    ko = torch.empty((1, 2, 128), device="cuda")
    vo = torch.empty((1, 2, 128), device="cuda")
    graph = torch.cuda.CUDAGraph()
    out3 = torch.zeros_like(ref)
    with torch.cuda.graph(graph):
        cache.reshape_and_cache(0, rows, rows, slot, 1)
        cache.gather_cached_rows(0, slot, 1, ko, vo)
        cache.paged_decode_attention(0, qd, hq, d_table, mb, d_lens, n, out3, ws)
    for seed in (1, 2):
        torch.manual_seed(seed)
        rows.copy_(torch.randn((1, 2, 128), device="cuda").bfloat16())
        graph.replay()
        torch.cuda.synchronize()
        got, gk = out3.clone(), ko.clone()
        cache.reshape_and_cache(0, rows, rows, slot, 1)
        cache.paged_decode_attention(0, qd, hq, d_table, mb, d_lens, n, out, ws)
        cache.gather_cached_rows(0, slot, 1, ko, vo)
        assert torch.equal(got, out) and torch.equal(gk, ko) and torch.equal(ko, vo)
    assert cache.kv_pool_device_status() == 0


@pytest.mark.parametrize("pinned", [False, True])
def test_whole_step_through_host_buffers(pinned):
    wl = q4_workload("q4_host", 4, 16, 71, [1, 16, 90, 333], fork=150, layers=2)
    orc = OracleRun(wl)
    cache, run = make(wl)
    for step in range(2):
        so, co, q, outs = orc.step(step)
        _, k, v = wl.step_values(step)
        n, hq, L = len(wl.decode_seqs), wl.n_q_heads, 2
        mb = max(-(-(run.lengths.get(s, 0) + 1) // 16) for s in wl.decode_seqs)
        host = lambda x: torch.from_numpy(np.ascontiguousarray(x).view(np.int16))  # noqa: E731
        hq_t, hk, hv = host(np.stack([q] * L)), host(k), host(v)
        ho = torch.empty((L, n, hq, 128), dtype=torch.float32)
        if pinned:
            hq_t, hk, hv, ho = (x.pin_memory() for x in (hq_t, hk, hv, ho))
        st = torch.empty(cache.kv_decode_step_staging_bytes(n, hq, mb), dtype=torch.uint8,
                         device="cuda")
        cache.kv_decode_step_host(wl.decode_seqs, hq, mb, hq_t, hk, hv, ho, st)
        for s in wl.decode_seqs:
            run.lengths[s] = run.lengths.get(s, 0) + 1
        for ly in range(L):
            assert max_err(ho.numpy()[ly], outs[ly]) <= step_tol(orc, q)
        assert same_pool(cache, orc.st)
    assert cache.kv_pool_device_status() == 0


def test_refusals():
    from paged_kv_cache_65_gb300 import KVError, PagedKVCache, _lib

    c = PagedKVCache(1, 8, 16, 2, 128, "q4_0")
    q = torch.zeros((1, 8, 128), dtype=torch.bfloat16, device="cuda")
    table = torch.zeros((1, 2), dtype=torch.int32, device="cuda")
    lens = torch.ones(1, dtype=torch.int32, device="cuda")
    out = torch.empty((1, 8, 128), device="cuda")
    ws = torch.empty(c.paged_decode_workspace_bytes(1, 8), dtype=torch.uint8, device="cuda")
    rows = torch.zeros((1, 2, 128), dtype=torch.bfloat16, device="cuda")

    def status(call):
        with pytest.raises(KVError) as e:
            call()
        return e.value.status

    c.kv_pool_set_option(_lib.KV_OPT_DECODE_PATH, 1)  # no CUDA-core pass over codes
    assert status(lambda: c.paged_decode_attention(0, q, 8, table, 2, lens, 1, out, ws)) == \
        _lib.KV_ERR_UNSUPPORTED
    c.kv_pool_set_option(_lib.KV_OPT_DECODE_PATH, 0)
    assert status(lambda: c.paged_decode_attention(0, q, 6, table, 2, lens, 1, out, ws)) == \
        _lib.KV_ERR_UNSUPPORTED  # three query heads per K/V head
    assert status(lambda: c.paged_decode_attention(0, q, 8, table, 2, lens, 1, out, ws[:64])) == \
        _lib.KV_ERR_INVALID_ARG
    c.seq_append_tokens(0, 1)
    h_plan, wsb = c.paged_decode_plan([0], 8, 2)
    d_plan = torch.from_numpy(h_plan).cuda()
    ws2 = torch.empty(wsb, dtype=torch.uint8, device="cuda")
    assert status(lambda: c.paged_decode_partials_planned_write(
        0, q, 8, rows, rows, table, 2, d_plan, h_plan, ws2)) == _lib.KV_ERR_UNSUPPORTED
    assert status(lambda: c.kv_pool_set_fp8_scales(1.0, 1.0)) == _lib.KV_ERR_INVALID_ARG
    with pytest.raises(TypeError):
        c.gather_cached_rows(0, lens, 1, out, out.bfloat16())
    c24 = PagedKVCache(1, 8, 24, 2, 128, "q4_0")  # 24 tokens: no pass
    assert status(lambda: c24.reshape_and_cache(0, rows, rows, lens.long(), 1)) == \
        _lib.KV_ERR_UNSUPPORTED
