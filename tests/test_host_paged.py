"""Host-side checks of the paged cache's entry points: sizes and refusals, no GPU needed."""
import ctypes

import pytest
import torch

import quantised_kv_long_gb300 as kvq

FAKE, BAD = 0x1000, 0x1004


def test_pool_size_is_the_block_footprint():
    for tk, tv in [("f16", "f16"), ("q8_0", "q8_0"), ("q8_0", "q4_0"), ("q4_0", "q4_0")]:
        for d in (128, 256):
            pool, state = kvq.paged_size(7, 48, 3, d, tk, tv)
            assert pool == 7 * 48 * 3 * d // 32 * (kvq.block_bytes(tk) + kvq.block_bytes(tv))
            assert state == 16
    # sizes past 32 bits
    pool, _ = kvq.paged_size(1 << 20, 64, 8, 128, "q4_0", "q4_0")
    assert pool == (1 << 20) * 64 * 8 * 4 * 36


@pytest.mark.parametrize("desc,status", [
    ((0, 16, 8, 128, "q8_0", "q8_0"), 1),            # no pages
    ((4, 0, 8, 128, "q8_0", "q8_0"), 1),             # empty pages
    ((4, 24, 8, 128, "q8_0", "q8_0"), 1),            # page size not a multiple of 16
    ((4, 16, 0, 128, "q8_0", "q8_0"), 1),            # no heads
    ((4, 16, 8, 64, "q8_0", "q8_0"), 2),             # head_dim
    ((4, 16, 8, 128, "q4_0", "q8_0"), 2),            # a pair that pages do not hold
    ((4, 16, 8, 128, "q5_1", "q5_1"), 2),
    ((4, 16, 8, 128, 9, 9), 2),
    ((2**31 - 1, 2**31 - 16, 2**31 - 1, 256, "f16", "f16"), 1),  # size overflow
])
def test_bad_descriptors(desc, status):
    with pytest.raises(kvq.KvqError) as e:
        kvq.paged_size(*desc)
    assert e.value.status == status


def test_null_and_misaligned_pointers():
    d = kvq.PagedDesc(4, 16, 2, 128, 1, 1)
    h = ctypes.c_void_p()
    L = kvq.lib
    assert L.kvq_paged_size(None, None, None) == 1
    assert L.kvq_paged_create(None, FAKE, FAKE, ctypes.byref(h)) == 1
    assert L.kvq_paged_create(ctypes.byref(d), None, FAKE, ctypes.byref(h)) == 1
    assert L.kvq_paged_create(ctypes.byref(d), FAKE, FAKE, None) == 1
    assert L.kvq_paged_create(ctypes.byref(d), BAD, FAKE, ctypes.byref(h)) == 4
    assert L.kvq_paged_create(ctypes.byref(d), FAKE, BAD, ctypes.byref(h)) == 4
    assert L.kvq_paged_destroy(None) == 1
    assert L.kvq_paged_read_error(None, None, None) == 1
    b = kvq.PagedBatch(1, 1, 1, 16, 0, FAKE, FAKE, 1, 1)
    assert L.kvq_paged_append(None, ctypes.byref(b), FAKE, FAKE, 0, 256, 256, None, None, 0, 0, None, 0, None) == 1
    assert L.kvq_paged_gather(None, ctypes.byref(b), FAKE, FAKE, 0, None) == 1
    sz = ctypes.c_size_t()
    assert L.kvq_paged_attention_workspace_size(None, ctypes.byref(b), 4, 0, ctypes.byref(sz)) == 1
    assert L.kvq_paged_attention(None, ctypes.byref(b), FAKE, 0, 4, 512, 1.0, FAKE, 1 << 20, FAKE, None, None) == 1


def fake_handle(types=(1, 1), dim=128):
    """A handle over addresses that are never touched: every refusal comes before a launch.
    The host struct, as kvq_paged_create fills it (descriptor, pool, state, device): without a GPU no
    device is current, so the handle is made by hand and the device check refuses the call at the latest."""
    class H(ctypes.Structure):
        _fields_ = [("desc", kvq.PagedDesc), ("pool", ctypes.c_void_p), ("state", ctypes.c_void_p), ("device", ctypes.c_int)]
    return H(kvq.PagedDesc(4, 16, 2, dim, *types), FAKE, FAKE, -2)


def batch(**kw):
    a = dict(n_seqs=2, n_tokens=5, max_q=4, max_len=32, cu_q=FAKE, lens=FAKE, block_table=FAKE, table_width=2, table_stride=2)
    a.update(kw)
    return kvq.PagedBatch(**a)


BAD_BATCHES = [(dict(n_seqs=-1), 1), (dict(n_tokens=-1), 1), (dict(max_q=0), 1), (dict(max_len=33), 1), (dict(max_len=-1), 1),
               (dict(table_width=0), 1), (dict(table_stride=1), 1), (dict(lens=0), 1), (dict(block_table=0), 1),
               (dict(cu_q=0, n_tokens=1), 1), (dict(lens=0x1002), 4), (dict(block_table=0x1001), 4), (dict(cu_q=0x1002), 4)]


@pytest.mark.parametrize("kw,status", BAD_BATCHES)
def test_bad_batches(kw, status):
    h, b, L = fake_handle(), batch(**kw), kvq.lib
    hp, bp, sz = ctypes.byref(h), ctypes.byref(b), ctypes.c_size_t()
    assert L.kvq_paged_append(hp, bp, FAKE, FAKE, 0, 256, 256, None, None, 0, 0, None, 0, None) == status
    assert L.kvq_paged_gather(hp, bp, FAKE, FAKE, 0, None) == status
    assert L.kvq_paged_attention_workspace_size(hp, bp, 4, 0, ctypes.byref(sz)) == status
    assert L.kvq_paged_attention(hp, bp, FAKE, 0, 4, 512, 1.0, FAKE, 1 << 20, FAKE, None, None) == status


def test_empty_batches_do_nothing():
    h, L = fake_handle(), kvq.lib
    for kw in (dict(n_seqs=0), dict(n_tokens=0)):
        b = batch(**kw)
        assert L.kvq_paged_append(ctypes.byref(h), ctypes.byref(b), FAKE, FAKE, 0, 256, 256, None, None, 0, 0, None, 0, None) == 0
        assert L.kvq_paged_gather(ctypes.byref(h), ctypes.byref(b), FAKE, FAKE, 0, None) == 0
        assert L.kvq_paged_attention(ctypes.byref(h), ctypes.byref(b), FAKE, 0, 4, 512, 1.0, FAKE, 0, FAKE, None, None) == 0


def rope(**kw):
    a = dict(cos_sin=FAKE, positions=0, n_positions=64, rot_dim=128, interleaved=0)
    a.update(kw)
    return kvq.RopeArgs(**a)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=3), 2), (dict(k=0), 1), (dict(v=0), 1), (dict(k=BAD), 4), (dict(v=BAD), 4), (dict(k_stride=248), 1),
    (dict(v_stride=248), 1), (dict(k_stride=260), 4), (dict(v_stride=257), 4), (dict(rope=rope(cos_sin=0)), 1),
    (dict(rope=rope(n_positions=0)), 1), (dict(rope=rope(rot_dim=0)), 1), (dict(rope=rope(rot_dim=12)), 1),
    (dict(rope=rope(rot_dim=136)), 1), (dict(rope=rope(cos_sin=BAD)), 4), (dict(rope=rope(positions=0x1002)), 4),
    (dict(q=FAKE), 1),                                                  # queries without a rotation
    (dict(q=FAKE, rope=rope(), n_q_heads=3), 1), (dict(q=FAKE, rope=rope(), n_q_heads=0), 1),
    (dict(q=FAKE, rope=rope(), q_out=0), 1), (dict(q=BAD, rope=rope()), 4), (dict(q=FAKE, rope=rope(), q_out=BAD), 4),
    (dict(q=FAKE, rope=rope(), q_stride=504), 1), (dict(q=FAKE, rope=rope(), q_out_stride=516), 4),
    (dict(q=FAKE, rope=rope(), q_out=FAKE, q_out_stride=520), 1),       # in place with another stride
])
def test_bad_appends(kw, status):
    a = dict(k=FAKE, v=FAKE, dtype=0, k_stride=256, v_stride=256, rope=None, q=0, n_q_heads=4, q_stride=512, q_out=0x2000,
             q_out_stride=512)
    a.update(kw)
    h, b = fake_handle(), batch()
    r = None if a["rope"] is None else ctypes.byref(a["rope"])
    assert kvq.lib.kvq_paged_append(ctypes.byref(h), ctypes.byref(b), a["k"], a["v"], a["dtype"], a["k_stride"], a["v_stride"], r,
                                    a["q"], a["n_q_heads"], a["q_stride"], a["q_out"], a["q_out_stride"], None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=3), 2), (dict(n_q_heads=3), 1), (dict(n_q_heads=0), 1), (dict(n_q_heads=65536), 2), (dict(q=0), 1), (dict(q=BAD), 4),
    (dict(q_stride=504), 1), (dict(q_stride=516), 4), (dict(out=0), 1), (dict(out=BAD), 4), (dict(workspace=0), 1),
    (dict(workspace=BAD), 4), (dict(lse=0x1002), 4),
    (dict(batch=batch(n_tokens=40, max_q=17), dtype=0), 2),  # fp32 queries: 16 per sequence
])
def test_bad_attention(kw, status):
    a = dict(q=FAKE, dtype=1, n_q_heads=4, q_stride=512, workspace=FAKE, out=FAKE, lse=0, batch=batch())
    a.update(kw)
    h = fake_handle()
    assert kvq.lib.kvq_paged_attention(ctypes.byref(h), ctypes.byref(a["batch"]), a["q"], a["dtype"], a["n_q_heads"], a["q_stride"],
                                       1.0, a["workspace"], 1 << 30, a["out"], a["lse"], None) == status


def test_bad_gathers():
    h, b = fake_handle(), batch()
    for k, v, dt, status in [(0, FAKE, 0, 1), (FAKE, 0, 0, 1), (BAD, FAKE, 0, 4), (FAKE, BAD, 0, 4), (FAKE, FAKE, 7, 2)]:
        assert kvq.lib.kvq_paged_gather(ctypes.byref(h), ctypes.byref(b), k, v, dt, None) == status


def test_another_device_is_refused():
    """A handle whose device is not current: refused after the other checks, nothing launched
    (without a GPU the runtime itself reports an error)."""
    h, b = fake_handle(), batch()
    want = 1 if torch.cuda.is_available() else 5
    assert kvq.lib.kvq_paged_gather(ctypes.byref(h), ctypes.byref(b), FAKE, FAKE, 0, None) == want
    assert kvq.lib.kvq_paged_append(ctypes.byref(h), ctypes.byref(b), FAKE, FAKE, 0, 256, 256, None, None, 0, 0, None, 0, None) == want
    assert kvq.lib.kvq_paged_attention(ctypes.byref(h), ctypes.byref(b), FAKE, 1, 4, 512, 1.0, FAKE, 1 << 30, FAKE, None, None) == want
    assert kvq.lib.kvq_paged_read_error(ctypes.byref(h), None, ctypes.byref(ctypes.c_int32())) == want


def test_binding_refuses_what_it_cannot_pass():
    """Host tensors and wrong types never reach the library."""
    c = object.__new__(kvq.PagedCache)
    c.device, c.page_size, c.n_kv_heads, c.head_dim, c.handle = torch.device("cpu"), 16, 2, 128, None
    t, n = torch.zeros((2, 3), dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    assert c._batch(t, n, None, None, None, 2).max_len == 48
    for bad in [dict(block_table=t.long()), dict(lens=n.long()), dict(block_table=t[:1]), dict(cu_q=torch.zeros(2, dtype=torch.int32)),
                dict(cu_q=torch.zeros(3)), dict(n_tokens=1)]:
        a = dict(block_table=t, lens=n, cu_q=None, max_q=None, max_len=None, n_tokens=2)
        a.update(bad)
        with pytest.raises(ValueError):
            c._batch(**a)
    x = torch.zeros((4, 2, 128), dtype=torch.float16)
    assert c._rows(x, 2, "k") == (x.data_ptr(), 256)
    for bad in [x[..., :64], x.double(), x.transpose(0, 1), x[:, :1], x[0], torch.zeros((4, 2, 256), dtype=torch.float16)[..., ::2]]:
        with pytest.raises(ValueError):
            c._rows(bad, 2, "k")
    fused = torch.zeros((4, 6, 128), dtype=torch.float16)
    assert c._rows(fused[:, 2:4], 2, "k") == (fused.data_ptr() + 2 * 128 * 2, 6 * 128)
    with pytest.raises(ValueError):
        kvq.Rope(torch.zeros((4, 8)))


def test_lengths_near_32_bits_are_refused():
    """Lengths are rounded up to whole blocks in 32 bits on the device."""
    h, L, sz = fake_handle(), kvq.lib, ctypes.c_size_t()
    for max_len, status in ((2**31 - 1, 2), (2**31 - 1024, 2)):
        b = batch(max_len=max_len, table_width=2**28, table_stride=2**28)
        assert L.kvq_paged_gather(ctypes.byref(h), ctypes.byref(b), FAKE, FAKE, 0, None) == status
        assert L.kvq_paged_attention_workspace_size(ctypes.byref(h), ctypes.byref(b), 4, 0, ctypes.byref(sz)) == status


def test_sizes_past_32_bits_do_not_wrap():
    for desc in ((2**32 + 1, 16, 2, 128), (4, 2**32 + 16, 2, 128), (4, 16, 2**32 + 2, 128), (4, 16, 2, 2**32 + 128)):
        with pytest.raises(ValueError):
            kvq.paged_size(*desc, "q8_0", "q8_0")
