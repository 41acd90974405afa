"""q4_0 pools without a GPU: creation's checks, refusals of device calls,
plans, and the oracle's q4_0 store."""

import ctypes as C

import numpy as np
import pytest

import synth
from oracle.kv_store import KVStore
from oracle.q4 import q4_decode, q4_encode


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_65_gb300 import _lib

    return _lib


def test_creation_checks_groups_and_chunk_alignment(lib):
    from paged_kv_cache_65_gb300 import KVError, PagedKVCache

    PagedKVCache(1, 8, 16, 2, 128, "q4_0", allocate=False)
    PagedKVCache(1, 8, 8, 1, 32, "q4_0", allocate=False)
    for B, D in ((16, 48), (16, 16), (4, 32), (1, 128), (2, 64), (12, 32)):
        # D no multiple of 32, or B * D / 16 scale bytes no multiple of 16
        with pytest.raises(KVError) as e:
            PagedKVCache(1, 8, B, 1, D, "q4_0", allocate=False)
        assert e.value.status == lib.KV_ERR_INVALID_ARG, (B, D)


def test_host_only_pools_refuse_device_calls(lib):
    from paged_kv_cache_65_gb300 import KVError, PagedKVCache

    c = PagedKVCache(1, 8, 16, 2, 128, "q4_0", allocate=False)
    calls = [lambda: c.reshape_and_cache(0, 16, 16, 16, 1),
             lambda: check(lib.lib.gather_cached_rows(c.handle, 0, 16, 1, 16, 16, 0, None)),
             lambda: check(lib.lib.paged_decode_partials(c.handle, 0, 16, 8, 16, 4, 16, 1, 0.0, 16,
                                                         1 << 30, None))]

    def check(st):
        lib.check(st)

    for call in calls:
        with pytest.raises(KVError) as e:
            call()
        assert e.value.status == lib.KV_ERR_INVALID_ARG


def test_gather_refuses_bad_arguments(lib):
    from paged_kv_cache_65_gb300 import PagedKVCache

    # aligned addresses that are never read: every call is refused on the host
    buf = (C.c_uint8 * 64)()
    a = (C.addressof(buf) + 15) & ~15
    c = PagedKVCache(2, 8, 16, 2, 128, "q4_0", allocate=False, k_cache=None)
    f = lib.lib.gather_cached_rows
    bad = lib.KV_ERR_INVALID_ARG
    assert f(None, 0, a, 1, a, a, 0, None) == bad
    assert f(c.handle, 0, a, -1, a, a, 0, None) == bad
    assert f(c.handle, 2, a, 1, a, a, 0, None) == bad
    assert f(c.handle, -2, a, 1, a, a, 0, None) == bad
    assert f(c.handle, 0, a, 1, a, a, 2, None) == bad        # FP8 outputs
    assert f(c.handle, 0, a, 1, a + 4, a, 0, None) == bad
    assert f(c.handle, 0, a, 1, a, a + 8, 1, None) == bad
    assert f(c.handle, 0, None, 1, a, a, 0, None) == bad
    assert f(c.handle, 0, a, 1, None, a, 0, None) == bad
    assert f(c.handle, 0, None, 0, None, None, 0, None) == lib.KV_OK


def test_device_tables_option(lib):
    from paged_kv_cache_65_gb300 import KVError, PagedKVCache

    c = PagedKVCache(1, 8, 16, 2, 128, "q4_0", allocate=False)
    c.kv_pool_set_option(lib.KV_OPT_DEVICE_TABLES, 1)
    c.kv_pool_set_option(lib.KV_OPT_DEVICE_TABLES, 0)
    for v in (-1, 2):
        with pytest.raises(KVError):
            c.kv_pool_set_option(lib.KV_OPT_DEVICE_TABLES, v)


@pytest.mark.parametrize("D,path,kernel", [(64, 0, 3), (64, 2, 2), (64, 3, 3), (128, 0, 3), (128, 2, 2), (128, 3, 3)])
def test_plans_follow_the_decode_path(lib, D, path, kernel):
    from paged_kv_cache_65_gb300 import PagedKVCache
    from paged_kv_cache_65_gb300.cache import parse_plan

    # three sharers of eight query heads a K/V head: 24 columns; 3 = the wide form
    c = PagedKVCache(1, 64, 16, 2, D, "q4_0", allocate=False)
    c.kv_pool_set_option(lib.KV_OPT_DECODE_PATH, path)
    c.seq_append_tokens(0, 512)
    for s in (1, 2, 3):
        c.seq_fork(0, s)
    c.seq_append_slots([1, 2, 3])
    buf, ws = c.paged_decode_plan([1, 2, 3], 16, 64)
    plan = parse_plan(buf)
    assert plan["kernel"] == kernel and plan["n_shared_segs"] > 0 and ws > 0


def test_oracle_store_round_trip():
    rng = np.random.default_rng(5)
    st = KVStore(1, 4, 8, 2, 64, "q4_0")
    assert st.K.shape == (1, 4, 8, 2, 32) and st.Ks.shape == (1, 4, 8, 2, 2)
    x = synth.storage_values(rng.standard_normal((2, 3, 2, 64)).astype(np.float32), "q4_0")
    st.reshape_and_cache(0, x[0], x[1], [9, -1, 31])
    st.copy_block(1, 2)
    f = (x.astype(np.uint32) << 16).view(np.float32)
    for name, i in (("K", 0), ("V", 1)):
        codes, sc = q4_encode(f[i])
        assert np.array_equal(getattr(st, name)[0, 1, 1], codes[0])
        assert np.array_equal(getattr(st, name)[0, 2, 1], codes[0])
        assert np.array_equal(getattr(st, name + "s")[0, 3, 7], sc[2])
    k, v = st.gather(0, [1], 2)
    assert np.array_equal(k[1], q4_decode(*q4_encode(f[0, 0])))
    assert np.array_equal(v[1], q4_decode(*q4_encode(f[1, 0])))
