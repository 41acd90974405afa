"""Chunked prefill over q4_0 pools on the GPU.

Two references in 64 bits.  Against attention over the fp16 copies (c d over
the power of two of the sequence and K/V head, rounded to fp16, times it) the
pass itself is held: its weights are fp16 (half a step, 2^-11 relative, 2^-25
absolute below 2^-14, p <= 2^8 with the largest weight of a row within a factor
2^8 of 1 or above it, so l >= 1 / (1 + 2^-7)), sums and scores are float32:
    2^-11 (1 + 2^-3) max|v| + T max|v| 2^-25 + 2 e_s ln 2 max|v|,
e_s as in the decode tests without the offset.  Against attention over c d
itself a copied value is off by 2^-11 relative, which adds 2^-11 max|v| for V
and, for K, a score error of at most 2^-11 max_{query, key} sum |q k| scale.
"""

import numpy as np
import pytest

import synth
from oracle.prefill import prefill_attention
from oracle.runner import OracleRun

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def prefill_wl(name, G, B, H, hist, chunk, seed, layers=1):
    n_blocks = sum(-(-(h + c) // B) for h, c in zip(hist, chunk)) + 7
    ops = [("append", s, h, s) for s, h in enumerate(hist) if h > 0]
    return synth.workloads.PrefillWorkload(name, layers, n_blocks, B, H * G, H, 128, "q4_0", seed,
                                           synth.permutation((seed, 0), n_blocks), ops,
                                           list(range(len(hist))), "", list(enumerate(chunk)))


def make(wl, fill=0):
    from paged_kv_cache_65_gb300 import PagedKVCache
    from paged_kv_cache_65_gb300.driver import DeviceRun

    cache = PagedKVCache(wl.n_layers, wl.n_blocks, wl.block_size, wl.n_kv_heads, wl.head_dim,
                         wl.dtype, free_order=wl.free_order)
    cache.k.fill_(fill)
    cache.v.fill_(fill)
    run = DeviceRun(cache, wl.n_q_heads)
    for op in wl.build_ops:
        run.apply(op, wl.append_values)
    return cache, run


def copied(x, scales):
    """The staged copy of one sequence's rows [T, H, D] in 64 bits: fp16 of
    x / 2^e times 2^e, e = floor(log2 max scale) - 11 per K/V head."""
    out = np.empty_like(x)
    for h in range(x.shape[1]):
        d = scales[:, h].view(np.float16).astype(np.float64).max()
        p = 2.0 ** (np.floor(np.log2(d)) - 11) if d > 0 else 1.0
        out[:, h] = (x[:, h] / p).astype(np.float16).astype(np.float64) * p
    return out


def check(wl, got, orc, q, layer=0, out_eps=0.0):
    qf = (np.asarray(q).astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    row = 0
    G, B, D = wl.n_q_heads // wl.n_kv_heads, wl.block_size, 128
    for s, c in wl.chunks:
        if c == 0:
            continue
        T = orc.bm.lengths[s]
        k, v = orc.st.gather(layer, orc.bm.tables[s], T)
        blocks = np.asarray(orc.bm.tables[s])[np.arange(T) // B]
        ks, vs = (a[layer, blocks, np.arange(T) % B] for a in (orc.st.Ks, orc.st.Vs))
        kc, vc = copied(k, ks), copied(v, vs)
        qs = qf[row:row + c]
        mine = got[row:row + c].astype(np.float64)
        v_max, scale = np.abs(v).max(), 1.4427 / np.sqrt(D)
        qk = max(float((np.abs(qs[:, h]) @ np.abs(k[:, h // G]).T).max()) for h in range(H_Q(wl)))
        e_s = 2.0**-24 * (D + 8) * qk * scale
        tol = (2.0**-11 * 1.125 + 2 * e_s * 0.6932 + T * 2.0**-25 + out_eps) * v_max
        ref = prefill_attention(qs, kc, vc)
        assert np.abs(mine - ref).max() <= tol, (s, c, T)
        tol += (2.0**-11 + 2 * 0.6932 * 2.0**-11 * qk * scale) * v_max
        assert np.abs(mine - prefill_attention(qs, k, v)).max() <= tol
        row += c


def H_Q(wl):
    return wl.n_q_heads


@pytest.mark.parametrize("G,B,H,hist,chunk", [
    (4, 16, 2, [0, 37, 200], [45, 130, 1]),
    (1, 8, 1, [0, 5, 127, 128], [1, 128, 129, 1]),
    (8, 32, 2, [300, 40, 63], [17, 0, 65]),
    (2, 64, 3, [0, 1000], [257, 33]),
    (4, 128, 1, [5, 260], [1, 100]),
    (2, 192, 2, [191, 192, 400], [1, 2, 70]),
    (1, 256, 1, [511], [300]),
])
@pytest.mark.parametrize("scheduled", [False, True])
def test_prefill_of_ragged_chunks(G, B, H, hist, chunk, scheduled):
    wl = prefill_wl("q4_prefill", G, B, H, hist, chunk, 50 + G + B)
    orc = OracleRun(wl)
    cache, run = make(wl, fill=0xFF)  # NaN scales in unused slots
    _, _, q = orc.prefill_step(0)
    _, k, v = wl.chunk_values(0)
    got = run.prefill_step(wl.chunks, q, k, v, scheduled=scheduled).cpu().numpy()[0]
    check(wl, got, orc, q)
    assert cache.kv_pool_device_status() == 0


def test_prefill_layers_and_bfloat16_outputs():
    wl = prefill_wl("q4_prefill2", 4, 16, 2, [20, 300], [100, 31], 77, layers=2)
    orc = OracleRun(wl)
    cache, run = make(wl)
    _, _, q = orc.prefill_step(0)
    _, k, v = wl.chunk_values(0)
    got = run.prefill_step(wl.chunks, q, k, v, out_dtype=torch.bfloat16).float().cpu().numpy()
    for layer in range(2):
        check(wl, got[layer], orc, q, layer, 2.0**-8)


@pytest.mark.parametrize("q_scale,k_scale,v_scale", [(1.0, 1e-5, 1e-5), (1e5, 1e-4, 3e4), (1e-5, 5e4, 1e-7)])
def test_prefill_magnitudes(q_scale, k_scale, v_scale):
    import dataclasses

    wl = prefill_wl("q4_prefill_mag", 4, 16, 2, [150], [70], 91)

    def scaled(x, f):
        y = (x.astype(np.uint32) << 16).view(np.float32) * np.float32(f)
        return synth.storage_values(y, "q4_0")

    class Scaled(type(wl)):
        def append_values(self, seed, n):
            k, v = super().append_values(seed, n)
            return scaled(k, k_scale), scaled(v, v_scale)

        def chunk_values(self, step):
            q, k, v = super().chunk_values(step)
            return scaled(q, q_scale), scaled(k, k_scale), scaled(v, v_scale)

    wl = Scaled(**{f.name: getattr(wl, f.name) for f in dataclasses.fields(wl)})
    orc = OracleRun(wl)
    cache, run = make(wl)
    _, _, q = orc.prefill_step(0)
    _, k, v = wl.chunk_values(0)
    got = run.prefill_step(wl.chunks, q, k, v).cpu().numpy()[0]
    check(wl, got, orc, q)
    assert cache.kv_pool_device_status() == 0


def test_prefill_flags_bad_blocks_and_reuses_its_workspace():
    from paged_kv_cache_65_gb300 import _lib

    wl = prefill_wl("q4_prefill_bad", 4, 16, 2, [40, 90], [8, 30], 13)
    orc = OracleRun(wl)
    cache, run = make(wl)
    _, _, q = orc.prefill_step(0)
    _, k, v = wl.chunk_values(0)
    got = run.prefill_step(wl.chunks, q, k, v)
    from paged_kv_cache_65_gb300.driver import to_device

    d_table, d_lens, mb = run.tables([0, 1])
    start = torch.tensor([0, 8, 38], dtype=torch.int32, device="cuda")
    ws = torch.empty(cache.paged_prefill_staging_bytes(2, mb), dtype=torch.uint8, device="cuda")
    out = torch.zeros_like(got[0])
    bad = d_table.clone()
    bad[0, 1] = cache.N
    bad[1, 0] = -5
    qd = to_device(q, "bf16", "cuda")
    cache.paged_prefill_attention_staged(0, qd, 8, bad, mb, start, d_lens, 2, out, ws, max_chunk=30)
    assert cache.kv_pool_device_status() == _lib.KV_DEV_BAD_BLOCK_ID
    # the same workspace, a smaller batch: rows of the other sequence stay
    out.fill_(7.0)
    cache.paged_prefill_attention_staged(0, qd[8:], 8, d_table[1:], mb, start[1:] - 8, d_lens[1:], 1,
                                         out[8:], ws, max_chunk=30)
    assert torch.equal(out[8:], got[0, 8:]) and bool((out[:8] == 7.0).all())
    assert cache.kv_pool_device_status() == 0


def test_prefill_refusals():
    from paged_kv_cache_65_gb300 import KVError, PagedKVCache, _lib

    def status(call):
        with pytest.raises(KVError) as e:
            call()
        return e.value.status

    t = torch.zeros((1, 2), dtype=torch.int32, device="cuda")
    lens = torch.ones(1, dtype=torch.int32, device="cuda")
    start = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    c = PagedKVCache(1, 8, 16, 2, 128, "q4_0")
    q = torch.zeros((1, 8, 128), dtype=torch.bfloat16, device="cuda")
    out = torch.empty((1, 8, 128), device="cuda")
    ws = torch.empty(c.paged_prefill_staging_bytes(1, 2), dtype=torch.uint8, device="cuda")
    assert status(lambda: c.paged_prefill_attention_staged(0, q, 8, t, 2, start, lens, 1, out,
                                                           ws[:256], max_chunk=1)) == \
        _lib.KV_ERR_INVALID_ARG
    assert status(lambda: c.paged_prefill_attention(0, q, 8, t, 2, start, lens, 1, 1, out)) == \
        _lib.KV_ERR_UNSUPPORTED  # read through a copy only
    assert status(lambda: c.paged_prefill_attention_staged(0, q, 6, t, 2, start, lens, 1, out, ws,
                                                           max_chunk=1)) == _lib.KV_ERR_UNSUPPORTED
    c64 = PagedKVCache(1, 8, 16, 2, 64, "q4_0")
    q64 = torch.zeros((1, 8, 64), dtype=torch.bfloat16, device="cuda")
    assert status(lambda: c64.paged_prefill_attention_staged(
        0, q64, 8, t, 2, start, lens, 1, torch.empty((1, 8, 64), device="cuda"), ws,
        max_chunk=1)) == _lib.KV_ERR_UNSUPPORTED
