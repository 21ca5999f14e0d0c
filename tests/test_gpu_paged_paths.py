"""Paged cache on the GPU: sizes and contents that take the kernels' rarer paths."""
import math

import numpy as np
import pytest
import torch

from tests.paged_ref import PAIRS, angles, attend, bounds, cumulative, dev, rotate, stored
from tests.test_gpu_paged import Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvq():
    import quantised_kv_long_gb300 as m
    return m


@pytest.mark.parametrize("pair", PAIRS)
@pytest.mark.parametrize("d,dtype,page", [(128, "bf16", 64), (128, "f16", 48), (256, "bf16", 48), (256, "f16", 128)])
def test_chunks_without_room_for_operands(kvq, pair, d, dtype, page):
    """A length bound whose 16-bit operands would pass the workspace's limit: they are made in the kernel."""
    lens, new = [130, 0, 700, 65, 1, 2000], [40, 0, 300, 65, 1, 17]
    b = Batch(kvq, lens, new, d=d, pair=pair, page=page, seed=21)
    width = (1 << 20) // page
    wide = torch.full((len(lens), width), -9, dtype=torch.int32, device="cuda")
    wide[:, :b.table.shape[1]] = b.table
    q = b.queries(8, dtype)
    kw = dict(cu_q=b.cu, max_q=300, return_lse=True)
    dt = q.dtype
    assert b.cache.workspace_bytes(len(lens), b.n, 8, width * page, 300, dt) < 2 ** 27
    small = b.cache.workspace_bytes(len(lens), b.n, 8, 2048, 300, dt)
    out, lse = b.cache.attention(q, wide, b.lens_t, max_len=width * page, **kw)
    b.check(q, dtype, out, lse)
    # the same call with a near bound takes the other way and meets the same bounds
    assert small > b.cache.workspace_bytes(len(lens), b.n, 8, width * page, 300, dt)
    out2, lse2 = b.cache.attention(q, b.table, b.lens_t, max_len=2048 if b.table.shape[1] * page >= 2048 else None, **kw)
    b.check(q, dtype, out2, lse2)
    assert b.cache.read_error() == 0


def test_more_chunks_than_one_launch_takes(kvq):
    rng = np.random.default_rng(31)
    new = rng.integers(9, 24, 300).tolist()
    new[7] = new[256] = new[299] = 0
    new[100] = 1  # and one for the kernel of few queries
    lens = [m + int(x) for m, x in zip(new, rng.integers(0, 90, 300))]
    b = Batch(kvq, lens, new, hkv=1, page=16, seed=5)
    q = b.queries(4, "bf16")
    out, lse = b.cache.attention(q, b.table, b.lens_t, cu_q=b.cu, max_q=max(new), return_lse=True)
    b.check(q, "bf16", out, lse)
    assert b.cache.read_error() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens,new", [([0, 1, 16, 100, 500], [1, 1, 1, 1, 1]), ([0, 3, 17, 900], [2, 5, 0, 1]), ([0], [3]), ([1000] * 76, [1] * 76)])
def test_short_contexts(kvq, lens, new, dtype):
    """Few short sequences, one unit of work each: none, one and several row groups, lengths of zero."""
    b = Batch(kvq, lens, new, hkv=2, pair=("q4_0", "q4_0"), page=16, seed=8)
    q = b.queries(12, dtype)
    out, lse = b.cache.attention(q, b.table, b.lens_t, cu_q=b.cu, max_q=max(new), return_lse=True)
    b.check(q, dtype, out, lse)
    assert b.cache.read_error() == 0


def test_offsets_that_overlap(kvq):
    """More tokens in the offsets than the call has: what does not fit is left out and reported."""
    n, length = 40, 320
    b = Batch(kvq, [length] * 12, [n] * 12, hkv=2, page=16, seed=4)
    cu = dev([0 if i % 2 == 0 else n for i in range(13)])
    q = b.queries(8, "bf16")[:n].contiguous()
    out = b.cache.attention(q, b.table, b.lens_t, cu_q=cu, max_q=n, max_len=length)
    assert b.cache.read_error() == kvq.DEVERR_BATCH
    assert torch.isfinite(out).all()


@pytest.mark.parametrize("pair", PAIRS)
def test_missing_angles_inside_a_tile(kvq, pair):
    """A chunk whose tile has a token without angles: that row is left as it was, the others are written."""
    n, rot = 64, 64
    table, lens = dev([[3, 0, 1, 2]]), dev([n])
    cache = kvq.PagedCache(4, 16, 2, 128, *pair)
    rng = np.random.default_rng(2)
    old = rng.standard_normal((n, 2, 128)).astype(np.float32)
    new = rng.standard_normal((n, 2, 128)).astype(np.float32)
    cu, cs = dev([0, n]), angles(64, rot)
    cache.append(torch.from_numpy(old).cuda(), torch.from_numpy(old).cuda(), table, lens, cu_q=cu, max_q=n)
    pos = np.arange(n)[::-1].copy()
    pos[[5, 33, 47]] = [-1, 64, 2 ** 31 - 1]
    q = torch.from_numpy(new).cuda()
    q_out = torch.full_like(q, 7.0)
    cache.append(q, q, table, lens, cu_q=cu, max_q=n, rope=kvq.Rope(torch.from_numpy(cs).cuda()), positions=dev(pos), q=q, q_out=q_out)
    assert cache.read_error() == kvq.DEVERR_BATCH
    k, v = cache.gather(table, lens, n, cu_q=cu, max_q=n, dtype=torch.float32)
    keep = np.zeros(n, bool)
    keep[[5, 33, 47]] = True
    turned = rotate(new, cs, np.where(keep, 0, pos), rot, False)
    want_k = np.where(keep[:, None, None], old, turned)
    want_v = np.where(keep[:, None, None], old, new)
    assert np.array_equal(k.cpu().numpy().astype(np.float64), stored(pair[0], want_k).astype(np.float32).astype(np.float64))
    assert np.array_equal(v.cpu().numpy().astype(np.float64), stored(pair[1], want_v).astype(np.float32).astype(np.float64))
    got = q_out.cpu().numpy()
    assert np.array_equal(got[~keep], turned[~keep]) and (got[keep] == 7.0).all()


@pytest.mark.parametrize("new", [8, 70])
def test_infinite_keys_behind_a_token(kvq, new):
    """Keys that overflow the cache's type reach the tokens that attend to them and no other."""
    length, bad = 200, 200 - 3
    b = Batch(kvq, [length], [new], pair=("f16", "f16"), page=16, seed=12)
    last = torch.from_numpy(b.k_rows[0][bad:bad + 1]).cuda()
    last[:, :, 0], last[:, :, 1] = 1e38, float("nan")
    value = torch.from_numpy(b.v_rows[0][bad:bad + 1]).cuda()
    b.cache.append(last, value, b.table, dev([bad + 1]))
    q = b.queries(4, "bf16")
    out = b.cache.attention(q, b.table, b.lens_t, cu_q=b.cu, max_q=new)
    k, v = b.values(0)
    o, _, av, qk = attend(q, k, v, 1 / math.sqrt(128))
    tol, _ = bounds(o, av, qk, "bf16", length, 128, True)
    free = new - 3  # tokens before the bad position
    assert ((out[:free].double() - o[:free]).abs() <= tol[:free]).all()
    assert not torch.isfinite(out[free:]).any()
    assert b.cache.read_error() == 0


def test_sizes_past_the_kernels_counts_are_refused(kvq):
    cache = kvq.PagedCache(4, 1 << 16, 1, 128, "q8_0", "q8_0")
    for n, heads, length in ((1 << 24, 64, 1 << 24), (1 << 30, 65535, 2 ** 31 - 2048)):
        with pytest.raises(kvq.KvqError) as e:
            cache.workspace_bytes(1, n, heads, length, n)
        assert e.value.status == 2
    # a prompt of a million tokens is within them
    assert cache.workspace_bytes(1, 1 << 20, 8, 1 << 20, 1 << 20) > 0
    assert cache.workspace_bytes(2 ** 30, 2 ** 30, 8, 1 << 20) > 0


def test_expanded_tables_are_refused(kvq):
    b = Batch(kvq, [40, 40], [1, 1], page=16)
    row = b.table[:1].expand(2, b.table.shape[1])
    with pytest.raises(kvq.KvqError) as e:
        b.cache.attention(b.queries(4, "bf16"), row, b.lens_t)
    assert e.value.status == 1


@pytest.mark.parametrize("pair", [("q8_0", "q4_0"), ("q4_0", "q4_0")])
@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("new", [1, 5])
def test_fp32_of_4_bit_pages_without_the_offset(kvq, pair, d, new):
    """fp32 outputs of 4-bit rows: the codes' offset adds no error of its own (the bounds of bounds() alone)."""
    lens = [700, 64, 3000]
    b = Batch(kvq, lens, [new] * 3, d=d, pair=pair, page=48, seed=15)
    q = b.queries(8, "f32")
    out = b.cache.attention(q, b.table, b.lens_t, cu_q=b.cu, max_q=new)
    at = 0
    for i, a in enumerate(lens):
        k, v = b.values(i)
        o, _, av, qk = attend(q[at:at + new], k, v, 1 / math.sqrt(d))
        tol, _ = bounds(o, av, qk, "f32", a, d, False)
        assert ((out[at:at + new].double() - o).abs() <= tol).all(), i
        # and in the norm, where roundings of 2^-22 of the weights and 2^-24 a step do not add up one way
        # (codes summed as subnormals, 0 .. 15, and the offset taken off after it gave 4.5e-6)
        err = (out[at:at + new].double() - o).norm() / o.norm()
        assert err < 2.0 ** -18, (i, float(err))
        at += new


@pytest.mark.parametrize("pair", PAIRS[1:])
@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("lift", [True, False])
def test_f16_chunks_keep_their_scores(kvq, pair, d, lift):
    """f16 activations over quantised pages: keys count as hi + lo, so the scores' part of the bound is 2^-20,
    not 2^-11 (lse has no other rounding of 16 bits)."""
    lens, new, page = [900, 130], [70, 130], 64
    b = Batch(kvq, lens, new, d=d, pair=pair, page=page, seed=16)
    width = b.table.shape[1] if lift else (1 << 21) // page
    wide = torch.full((2, width), -9, dtype=torch.int32, device="cuda")
    wide[:, :b.table.shape[1]] = b.table
    q = b.queries(8, "f16")
    out, lse = b.cache.attention(q, wide, b.lens_t, cu_q=b.cu, max_q=130, return_lse=True)
    at = 0
    for i, (a, m) in enumerate(zip(lens, new)):
        k, v = b.values(i)
        o, z, av, qk = attend(q[at:at + m], k, v, 1 / math.sqrt(d))
        tol, ltol = bounds(o, av, qk, "f16", a, d, False)
        assert ((out[at:at + m].double() - o).abs() <= tol).all(), i
        assert ((lse[at:at + m].double() - z).abs() <= ltol).all(), i
        at += m
    assert b.cache.read_error() == 0


def test_lengths_past_32_bits(kvq):
    """A table that stands for more positions than 32 bits count: the default bound is cut, a given one refused."""
    page, width = 1 << 16, 1 << 15
    cache = kvq.PagedCache(2, page, 1, 128, "q4_0", "q4_0")
    table = torch.full((1, width), 1, dtype=torch.int32, device="cuda")
    x = torch.randn((3, 1, 128), device="cuda")
    cu = dev([0, 3])
    cache.append(x, x, table, dev([3]), cu_q=cu, max_q=3)
    k, _ = cache.gather(table, dev([3]), 3, cu_q=cu, max_q=3, dtype=torch.float32)
    assert np.array_equal(k.cpu().numpy().astype(np.float64), stored("q4_0", x.cpu().numpy()))
    assert cache.read_error() == 0
    with pytest.raises(ValueError):
        cache.append(x, x, table, dev([3]), cu_q=cu, max_q=3, max_len=2 ** 32 + 16)
    with pytest.raises(ValueError):
        cache.attention(x, table, dev([3]), cu_q=cu, max_q=2 ** 32 + 3)
    with pytest.raises(ValueError):
        cache.workspace_bytes(1, 2 ** 32 + 1, 1, 64)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("hkv,hq", [(1, 128), (3, 300), (2, 2)])
def test_many_and_single_heads_per_kv_head(kvq, hkv, hq, dtype):
    """128, 100 and 1 query heads per KV head: one token fills the chunk kernel's rows, or 57 tokens do."""
    lens, new = [333, 90, 70, 1, 0], [3, 90, 1, 1, 2]
    b = Batch(kvq, lens, new, hkv=hkv, pair=("q8_0", "q4_0"), page=32, seed=23, pad=4)
    q = b.queries(hq, dtype)
    out, lse = torch.full_like(q, 5.0), None
    out, lse = b.cache.attention(q, b.table, b.lens_t, cu_q=b.cu, max_q=90, return_lse=True, out=out)
    b.check(q, dtype, out, lse)
    assert bool((out[b.n:] == 5.0).all())
    assert b.cache.read_error() == 0


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_one_sequence_of_any_tokens_in_a_captured_call(kvq, dtype):
    """A captured call of one sequence with a bound of 96 tokens, replayed for 96, 1, 0 and 17 of them; twice the
    same bits."""
    b = Batch(kvq, [400], [96], pair=("q8_0", "q8_0"), page=64, seed=24)
    q = b.queries(8, dtype)
    lens, cu = b.lens_t.clone(), b.cu.clone()
    out = torch.zeros_like(q)
    ws = torch.empty(b.cache.workspace_bytes(1, 96, 8, b.table.shape[1] * 64, 96, q.dtype), dtype=torch.uint8, device="cuda")
    run = lambda: b.cache.attention(q, b.table, lens, cu_q=cu, max_q=96, out=out, workspace=ws)  # noqa: E731
    run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    k, v = b.values(0)
    for n, length in ((96, 400), (1, 400), (0, 0), (17, 17), (96, 130), (2, 1)):
        lens.fill_(length)
        cu.copy_(dev([0, n]))
        got = []
        for _ in range(2):
            out.fill_(3.0)
            ws.fill_(0xff)  # nothing is kept from a call to the next
            g.replay()
            torch.cuda.synchronize()
            got.append(out.clone())
        assert torch.equal(got[0], got[1])
        o, _, av, qk = attend(q[:n], k[:length], v[:length], 1 / math.sqrt(128))
        if n:
            tol, _ = bounds(o, av, qk, dtype, length, 128, True)
            assert ((got[0][:n].double() - o).abs() <= tol).all(), (n, length)
        assert bool((got[0][n:] == 3.0).all()), (n, length)
    assert b.cache.read_error() == 0
