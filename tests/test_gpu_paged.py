"""Paged cache on the GPU: append with rotation, gather and attention through the public entry
points, against the CPU oracle's stored values and attention in 64 bits."""
import math

import numpy as np
import pytest
import torch

from tests import kvq_layout
from tests.paged_ref import DT, PAIRS, angles, attend, bounds, cumulative, dev, offset_terms, rotate, stored, table

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvq():
    import quantised_kv_long_gb300 as m
    return m


class Batch:
    """A paged cache filled with normal rows (outlier channels in the keys), and its plain twin."""

    def __init__(self, kvq, lens, new, hkv=2, d=128, pair=("q8_0", "q4_0"), page=32, seed=0, pad=0, max_len=None):
        rng = np.random.default_rng(seed)
        self.kvq, self.lens, self.new, self.hkv, self.d, self.pair, self.page = kvq, list(lens), list(new), hkv, d, pair, page
        self.table_np, self.pages = table(rng, lens, page)
        self.cache = kvq.PagedCache(self.pages, page, hkv, d, *pair)
        self.cache.pool.fill_(0xff)  # stale rows and scales: NaN bits
        self.k_rows = [rng.standard_normal((a, hkv, d)).astype(np.float32) for a in lens]
        self.v_rows = [rng.standard_normal((a, hkv, d)).astype(np.float32) for a in lens]
        for k in self.k_rows:
            k[:, :, 3::37] *= 5
        self.table, self.lens_t = dev(self.table_np), dev(self.lens)
        cu = dev(cumulative(lens))
        if sum(lens):
            self.cache.append(torch.from_numpy(np.concatenate(self.k_rows)).cuda(), torch.from_numpy(np.concatenate(self.v_rows)).cuda(),
                              self.table, self.lens_t, cu_q=cu, max_q=max(lens))
        self.cu = dev(cumulative(new))
        self.n = sum(new)
        self.n_pad = self.n + pad

    def values(self, b):
        return (torch.from_numpy(stored(self.pair[0], self.k_rows[b])).cuda(), torch.from_numpy(stored(self.pair[1], self.v_rows[b])).cuda())

    def queries(self, hq, dtype, seed=1):
        g = torch.Generator().manual_seed(seed)
        return torch.randn((self.n_pad, hq, self.d), generator=g).to(DT[dtype]).cuda()

    def check(self, q, dtype, out, lse, scale=None):
        """out and lse of every sequence's tokens against 64 bits, within the derived bounds."""
        scale = 1 / math.sqrt(self.d) if scale is None else scale
        at = 0
        for b, (a, m) in enumerate(zip(self.lens, self.new)):
            if m == 0:
                continue
            k, v = self.values(b)
            o, z, av, qk = attend(q[at:at + m], k, v, scale)
            tol, ltol = bounds(o, av, qk, dtype, a, self.d, dtype != "f32", offset_terms(self.pair, q[at:at + m], k, v, scale, a))
            got = out[at:at + m].double()
            assert torch.isfinite(got).all(), b
            worst = ((got - o).abs() / tol).max().item()
            assert worst <= 1, (b, worst)
            if lse is not None:
                zero = z == -math.inf
                assert torch.equal(lse[at:at + m] == -math.inf, zero)
                err = torch.where(zero, torch.zeros_like(z), lse[at:at + m].double() - z).abs()
                assert (err <= ltol).all(), (b, (err / ltol).max().item())
            at += m


def natural(cache, tk, tv, hkv, d, page, pages):
    """Dequantised pool, read by the documented layout on the host: two arrays [pages * page, hkv, d]."""
    pool = cache.pool.cpu().numpy().reshape(pages, hkv, page // 16, -1)
    ns = d // 128
    size = {t: kvq_layout.CODE_TILE[t] for t in (tk, tv)}
    kc, vc = size[tk] * ns, size[tv] * ns
    ks = 0 if tk == "f16" else 128 * ns
    parts = np.split(pool, [kc, kc + vc, kc + vc + ks], axis=-1)
    out = []
    for codes, scales, t, is_v in ((parts[0], parts[2], tk, False), (parts[1], parts[3], tv, True)):
        c, s = kvq_layout.decode_plane(np.ascontiguousarray(codes).reshape(-1), np.ascontiguousarray(scales).reshape(-1), t, is_v,
                                       pages, hkv, page, d)
        import oracle
        out.append(oracle.dequantize(t, c, s, d).transpose(0, 2, 1, 3).reshape(pages * page, hkv, d))
    return out


@pytest.mark.parametrize("pair", PAIRS)
@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_append_and_gather(kvq, pair, d, dtype):
    """Ragged appends that start and end anywhere in tiles and pages: the stored values are the
    oracle's to the bit, earlier rows and other pages keep theirs, and queries come back rotated."""
    rng = np.random.default_rng(d + len(dtype))
    hkv, hq, page, rot = 3, 6, 48, d
    lens, new = [1, 16, 77, 200, 0, 95, 300], [1, 16, 30, 1, 0, 50, 300]
    tab, pages = table(rng, lens, page)
    cache = kvq.PagedCache(pages, page, hkv, d, *pair)
    cache.pool.fill_(0x5a)
    before = cache.pool.clone()
    ang = angles(max(lens), rot)
    rope = kvq.Rope(torch.from_numpy(ang).cuda())
    # first the older rows, then the new ones
    old = [a - m for a, m in zip(lens, new)]
    rows = {}
    for step, (upto, count) in enumerate([(old, old), (lens, new)]):
        n = sum(count)
        k = torch.from_numpy(rng.standard_normal((n, hkv, d)).astype(np.float32) * 2).to(DT[dtype]).cuda()
        v = torch.from_numpy(rng.standard_normal((n, hkv, d)).astype(np.float32)).to(DT[dtype]).cuda()
        q = torch.from_numpy(rng.standard_normal((n, hq, d)).astype(np.float32)).to(DT[dtype]).cuda()
        r = cache.append(k, v, dev(tab), dev(upto), cu_q=dev(cumulative(count)), max_q=max(count), rope=rope, q=q)
        pos = np.concatenate([np.arange(a - m, a) for a, m in zip(upto, count)])
        kr = rotate(k.float().cpu().numpy(), ang, pos, rot, False)
        qr = torch.from_numpy(rotate(q.float().cpu().numpy(), ang, pos, rot, False)).to(DT[dtype])
        assert torch.equal(r.cpu(), qr)
        at = 0
        for b, m in enumerate(count):
            rows.setdefault(b, []).append((kr[at:at + m], v[at:at + m].float().cpu().numpy()))
            at += m
    k, v = cache.gather(dev(tab), dev(lens), sum(lens), cu_q=dev(cumulative(lens)), max_q=max(lens), dtype=torch.float32)
    want = [np.concatenate([np.concatenate([x[i] for x in rows[b]]) for b in range(len(lens))]) for i in (0, 1)]
    assert np.array_equal(k.cpu().numpy().astype(np.float64), stored(pair[0], want[0]))
    assert np.array_equal(v.cpu().numpy().astype(np.float64), stored(pair[1], want[1]))
    for kind in ("f16", "bf16"):
        k2, v2 = cache.gather(dev(tab), dev(lens), sum(lens), cu_q=dev(cumulative(lens)), max_q=max(lens), dtype=DT[kind])
        assert torch.equal(k2, k.to(DT[kind])) and torch.equal(v2, v.to(DT[kind]))
    # the documented layout, and pages of no sequence untouched
    nk, nv = natural(cache, *pair, hkv, d, page, pages)
    at = 0
    for b, a in enumerate(lens):
        slots = [tab[b, t // page] * page + t % page for t in range(a)]
        assert np.array_equal(nk[slots], stored(pair[0], want[0][at:at + a]))
        assert np.array_equal(nv[slots], stored(pair[1], want[1][at:at + a]))
        at += a
    used = set(tab[tab >= 0].tolist())
    free = [i for i in range(pages) if i not in used]
    view = cache.pool.view(pages, -1)
    assert free and torch.equal(view[free], before.view(pages, -1)[free])
    assert cache.read_error() == 0


@pytest.mark.parametrize("rot,interleaved", [(8, False), (64, False), (64, True), (96, False), (128, True), (24, True)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rotation_kinds(kvq, rot, interleaved, dtype):
    """Partial and interleaved rotations, given positions, strided inputs and rotation in place."""
    rng = np.random.default_rng(rot)
    hkv, hq, d, page = 2, 4, 128, 16
    lens, new = [40, 5], [33, 5]
    tab, pages = table(rng, lens, page)
    cache = kvq.PagedCache(pages, page, hkv, d, "f16", "f16")
    ang = angles(500, rot)
    rope = kvq.Rope(torch.from_numpy(ang).cuda(), interleaved=interleaved)
    pos = rng.integers(0, 500, sum(new)).astype(np.int32)
    fused = torch.from_numpy(rng.standard_normal((sum(new), hq + 2 * hkv, d)).astype(np.float32)).to(DT[dtype]).cuda()
    q, k, v = fused[:, :hq], fused[:, hq:hq + hkv], fused[:, hq + hkv:]
    want_q = torch.from_numpy(rotate(q.float().cpu().numpy(), ang, pos, rot, interleaved)).to(DT[dtype])
    want_k = rotate(k.float().cpu().numpy(), ang, pos, rot, interleaved)
    kv_before = fused[:, hq:].clone()
    r = cache.append(k, v, dev(tab), dev(lens), cu_q=dev(cumulative(new)), max_q=max(new), rope=rope, positions=dev(pos), q=q, q_out=q)
    assert r.data_ptr() == q.data_ptr() and torch.equal(q.cpu(), want_q) and torch.equal(fused[:, hq:], kv_before)
    gk, gv = cache.gather(dev(tab), dev(lens), sum(new), cu_q=dev(cumulative(new)), max_q=max(new), dtype=torch.float32)
    assert np.array_equal(gk.cpu().numpy(), stored("f16", want_k).astype(np.float32))
    assert np.array_equal(gv.cpu().numpy(), stored("f16", kv_before[:, hkv:].float().cpu().numpy()).astype(np.float32))
    assert cache.read_error() == 0


def test_append_single_tokens_without_cu_q(kvq):
    rng = np.random.default_rng(5)
    lens = [1, 17, 16, 64, 33]
    tab, pages = table(rng, lens, 16)
    cache = kvq.PagedCache(pages, 16, 8, 128, "q8_0", "q4_0")
    k = torch.randn((7, 8, 128), device="cuda")  # two padding rows behind the sequences
    v = torch.randn((7, 8, 128), device="cuda")
    ang = angles(64, 128)
    q = torch.randn((7, 16, 128), device="cuda")
    q_out = torch.full_like(q, 7.0)
    cache.append(k, v, dev(tab), dev(lens), rope=kvq.Rope(torch.from_numpy(ang).cuda()), q=q, q_out=q_out)
    pos = np.array(lens) - 1
    assert torch.equal(q_out[:5].cpu(), torch.from_numpy(rotate(q[:5].cpu().numpy(), ang, pos, 128, False)))
    assert bool((q_out[5:] == 7.0).all())
    gk, gv = cache.gather(dev(tab), dev(lens), 5, dtype=torch.float32)
    assert np.array_equal(gk.cpu().numpy().astype(np.float64), stored("q8_0", rotate(k[:5].cpu().numpy(), ang, pos, 128, False)))
    assert np.array_equal(gv.cpu().numpy().astype(np.float64), stored("q4_0", v[:5].cpu().numpy()))


def test_many_sequences(kvq):
    """Token lookup over more sequences than one round of the search covers, many of them empty."""
    rng = np.random.default_rng(9)
    new = rng.integers(0, 4, 1500)
    new[rng.random(1500) < 0.4] = 0
    lens = new + rng.integers(0, 20, 1500)
    new, lens = new.tolist(), lens.tolist()
    b = Batch(kvq, lens, new, hkv=1, pair=("q4_0", "q4_0"), page=16, seed=3)
    k, v = b.cache.gather(b.table, b.lens_t, b.n, cu_q=b.cu, max_q=3, dtype=torch.float32)
    want = np.concatenate([x[a - m:] if m else x[:0] for x, a, m in zip(b.k_rows, lens, new)])
    assert np.array_equal(k.cpu().numpy().astype(np.float64), stored("q4_0", want))
    q = b.queries(4, "bf16")
    out, lse = b.cache.attention(q, b.table, b.lens_t, cu_q=b.cu, max_q=3, return_lse=True)
    b.check(q, "bf16", out, lse)
    assert b.cache.read_error() == 0


@pytest.mark.parametrize("pair", PAIRS)
@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_attention_single_tokens(kvq, pair, d, dtype):
    """One token per sequence, lengths from none to several thousand positions, ends anywhere."""
    lens = [1, 2, 15, 16, 17, 31, 33, 255, 0, 1000, 2311]
    b = Batch(kvq, lens, [1] * len(lens), hkv=2, d=d, pair=pair, page=48, seed=d)
    q = b.queries(10, dtype)
    out, lse = b.cache.attention(q, b.table, b.lens_t, return_lse=True)
    b.check(q, dtype, out, lse)
    assert bool((out[8] == 0).all()) and bool((lse[8] == -math.inf).all())
    assert b.cache.read_error() == 0


@pytest.mark.parametrize("g", [1, 2, 3, 7, 8, 9, 16, 24])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attention_head_groups(kvq, g, dtype):
    lens = [700, 37]
    b = Batch(kvq, lens, [1, 1], hkv=3, pair=("q4_0", "q4_0"), page=16, seed=g)
    q = b.queries(3 * g, dtype)
    out, lse = b.cache.attention(q, b.table, b.lens_t, return_lse=True)
    b.check(q, dtype, out, lse)


@pytest.mark.parametrize("pair", PAIRS)
@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attention_drafts(kvq, pair, d, dtype):
    """A few tokens per sequence, causal among themselves; some sequences have none, one has more
    tokens than positions (its first tokens see nothing)."""
    lens, new = [5, 600, 16, 333, 4, 0, 3], [5, 16, 1, 7, 9, 0, 0]
    b = Batch(kvq, lens, new, hkv=2, d=d, pair=pair, page=16, seed=2)
    q = b.queries(8, dtype)
    out, lse = b.cache.attention(q, b.table, b.lens_t, cu_q=b.cu, max_q=16, return_lse=True)
    b.check(q, dtype, out, lse)
    assert bool((out[29:34] == 0).all()) and bool((lse[29:34] == -math.inf).all())


@pytest.mark.parametrize("pair", PAIRS)
@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_attention_chunks(kvq, pair, d, dtype):
    """Prompt chunks of odd sizes beside single tokens, over pages of odd sizes."""
    lens, new = [130, 1000, 64, 1, 517, 0, 300], [130, 257, 1, 1, 100, 0, 300]
    b = Batch(kvq, lens, new, hkv=2, d=d, pair=pair, page=80, seed=4)
    q = b.queries(10, dtype)
    out, lse = b.cache.attention(q, b.table, b.lens_t, cu_q=b.cu, max_q=300, return_lse=True)
    b.check(q, dtype, out, lse)
    assert b.cache.read_error() == 0


@pytest.mark.parametrize("g", [1, 3, 5, 8, 16])
def test_attention_chunk_head_groups(kvq, g):
    lens, new = [400, 61], [211, 61]
    b = Batch(kvq, lens, new, hkv=2, pair=("q8_0", "q4_0"), page=32, seed=g)
    q = b.queries(2 * g, "bf16")
    out, lse = b.cache.attention(q, b.table, b.lens_t, cu_q=b.cu, max_q=211, return_lse=True)
    b.check(q, "bf16", out, lse)


@pytest.mark.parametrize("scale", [0.0, -0.05, 0.3])
@pytest.mark.parametrize("new", [1, 40])
def test_attention_scales(kvq, scale, new):
    b = Batch(kvq, [300], [new], pair=("q8_0", "q8_0"), seed=7)
    q = b.queries(4, "bf16") * 0.25
    out, lse = b.cache.attention(q, b.table, b.lens_t, cu_q=b.cu, max_q=new, scale=scale, return_lse=True)
    b.check(q, "bf16", out, lse, scale=scale)


@pytest.mark.parametrize("new", [1, 70])
@pytest.mark.parametrize("magnitude", [1e-30, 1e-6, 1e5, 1e30])
def test_attention_query_range(kvq, new, magnitude):
    """bf16 queries outside float16's range: the scale brings the scores back."""
    b = Batch(kvq, [200], [new], pair=("q4_0", "q4_0"), seed=8)
    q = (b.queries(4, "f32") * magnitude).to(torch.bfloat16)
    out, lse = b.cache.attention(q, b.table, b.lens_t, cu_q=b.cu, max_q=new, scale=0.05 / magnitude, return_lse=True)
    b.check(q, "bf16", out, lse, scale=0.05 / magnitude)


@pytest.mark.parametrize("new", [1, 70])
@pytest.mark.parametrize("pair", [("q8_0", "q8_0"), ("q4_0", "q4_0")])
@pytest.mark.parametrize("k_mag,v_mag", [(3e5, 1.0), (1.0, 2e5), (1e-4, 1e-4)])
def test_attention_value_range(kvq, new, pair, k_mag, v_mag):
    """Stored values past float16's largest (a float16 scale times a code) and small ones."""
    rng = np.random.default_rng(1)
    if pair[0] == "q4_0":
        # q4_0 stores at most 8 x 65504 = 524,032; normal rows of 3e5 reach 4 x 3e5, whose scale
        # (150,000) is no float16: a third of that stays in the type and past 65504
        k_mag, v_mag = min(k_mag, 1e5), min(v_mag, 1e5)
    lens = [150]
    tab, pages = table(rng, lens, 32)
    cache = kvq.PagedCache(pages, 32, 2, 128, *pair)
    k = (rng.standard_normal((150, 2, 128)) * k_mag).astype(np.float32)
    v = (rng.standard_normal((150, 2, 128)) * v_mag).astype(np.float32)
    cache.append(torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), dev(tab), dev(lens), cu_q=dev([0, 150]), max_q=150)
    q = torch.randn((new, 4, 128), generator=torch.Generator().manual_seed(3)).cuda().bfloat16()
    scale = 0.05 / k_mag
    out, lse = cache.attention(q, dev(tab), dev(lens), cu_q=dev([0, new]), max_q=new, scale=scale, return_lse=True)
    ks, vs = (torch.from_numpy(stored(t, x)).cuda() for t, x in zip(pair, (k, v)))
    o, z, av, qk = attend(q, ks, vs, scale)
    tol, ltol = bounds(o, av, qk, "bf16", 150, 128, True, offset_terms(pair, q, ks, vs, scale, 150))
    if v_mag < 1:  # 16-bit values below 2^-14 are rounded absolutely, by 2^-25 each, summed with weights of at most 1
        tol = tol + 2.0 ** -24
    assert ((out.double() - o).abs() <= tol).all()
    assert ((lse.double() - z).abs() <= ltol).all()


@pytest.mark.parametrize("new", [1, 50])
def test_padding_rows_stay(kvq, new):
    b = Batch(kvq, [90, 200], [new, min(new, 3)], seed=3, pad=5)
    q = b.queries(4, "f16")
    q[b.n:] = float("nan")
    out = torch.full_like(q, 7.0)
    b.cache.attention(q, b.table, b.lens_t, cu_q=b.cu, max_q=new, out=out)
    b.check(q, "f16", out, None)
    assert bool((out[b.n:] == 7.0).all())


@pytest.mark.parametrize("new", [1, 12, 40])
def test_broken_entries_are_reported(kvq, new):
    """Sequences and pages that contradict the call: the error word says so, the other sequences'
    results are right, nothing outside the pool or the outputs is touched."""
    lens = [200, 100, 150, 120]
    counts = [new] * 4
    b = Batch(kvq, lens, counts, pair=("q8_0", "q8_0"), page=16, seed=6)
    q = b.queries(4, "bf16")

    def others(out, skip):
        at = 0
        for i, m in enumerate(counts):
            if i not in skip:
                k, v = b.values(i)
                o, _, av, qk = attend(q[at:at + m], k, v, 1 / math.sqrt(128))
                tol, _ = bounds(o, av, qk, "bf16", lens[i], 128, True)
                assert ((out[at:at + m].double() - o).abs() <= tol).all(), i
            at += m

    def run(**kw):
        a = dict(block_table=b.table, lens=b.lens_t, cu_q=b.cu, max_q=new)
        a.update(kw)
        return b.cache.attention(q, **a)

    for bad_len in (-1, b.table.shape[1] * 16 + 1, 2 ** 31 - 1):
        lens_t = b.lens_t.clone()
        lens_t[1] = bad_len
        others(run(lens=lens_t), {1})
        assert b.cache.read_error() == kvq.DEVERR_BATCH
        assert b.cache.read_error() == 0
    for bad_page in (-1, b.pages, 2 ** 31 - 1, -2 ** 31):
        t = b.table.clone()
        t[2, 3] = bad_page
        out = run(block_table=t)
        others(out, {2})
        assert torch.isfinite(out).all()
        assert b.cache.read_error() == kvq.DEVERR_BATCH
        # the same page in an append and a gather: the rows are not written, and read as zeros
        before = b.cache.pool.clone()
        cu = dev(cumulative(lens))
        k = torch.from_numpy(np.concatenate(b.k_rows)).cuda()
        v = torch.from_numpy(np.concatenate(b.v_rows)).cuda()
        b.cache.append(k, v, t, b.lens_t, cu_q=cu, max_q=200)
        assert torch.equal(before, b.cache.pool) and b.cache.read_error() == kvq.DEVERR_BATCH
        gk, _ = b.cache.gather(t, b.lens_t, sum(lens), cu_q=cu, max_q=200, dtype=torch.float32)
        assert bool((gk[300 + 48:300 + 64] == 0).all()) and bool((gk[300:300 + 48] != 0).any())
        assert b.cache.read_error() == kvq.DEVERR_BATCH
    # more tokens than max_q, and offsets that run backwards or past the tokens
    for cu in ([0, new + 1, 2 * new, 3 * new, 4 * new], [0, new, new - 1, 3 * new, 4 * new], [0, new, 2 * new, 3 * new, 4 * new + 9],
               [0, -5, 2 * new, 3 * new, 4 * new], [0, new, 2 * new, 3 * new, 2 ** 31 - 1]):
        out = torch.zeros_like(q)
        run(cu_q=dev(cu), out=out)
        assert b.cache.read_error() == kvq.DEVERR_BATCH, cu
        assert torch.isfinite(out).all()


def test_positions_outside_the_angles(kvq):
    cache = kvq.PagedCache(4, 16, 1, 128, "q8_0", "q8_0")
    cache.pool.zero_()
    rope = kvq.Rope(torch.from_numpy(angles(10, 128)).cuda())
    k = torch.randn((3, 1, 128), device="cuda")
    for pos in ([0, 10, 9], [-1, 0, 2 ** 31 - 1]):
        cache.pool.zero_()
        cache.append(k, k, dev([[0, 1]]), dev([3]), cu_q=dev([0, 3]), max_q=3, rope=rope, positions=dev(pos))
        gk, _ = cache.gather(dev([[0, 1]]), dev([3]), 3, cu_q=dev([0, 3]), max_q=3, dtype=torch.float32)
        for i, p in enumerate(pos):
            assert bool((gk[i] != 0).any()) == (0 <= p < 10)
        assert cache.read_error() == kvq.DEVERR_BATCH


def test_negative_positions_are_not_written(kvq):
    """More tokens than positions: the first tokens are padding in front, not an error."""
    cache = kvq.PagedCache(2, 16, 1, 128, "f16", "f16")
    k = torch.randn((6, 1, 128), device="cuda")
    cache.append(k, k, dev([[1]]), dev([4]), cu_q=dev([0, 6]), max_q=6)
    gk, _ = cache.gather(dev([[1]]), dev([4]), 6, cu_q=dev([0, 6]), max_q=6, dtype=torch.float32)
    assert bool((gk[:2] == 0).all()) and torch.equal(gk[2:], k[2:].half().float())
    assert cache.read_error() == 0


@pytest.mark.parametrize("new", [1, 64])
def test_shared_pages_and_strided_tables(kvq, new):
    """Two sequences with a common prefix share its pages; the table is a slice of a wider one."""
    rng = np.random.default_rng(0)
    cache = kvq.PagedCache(12, 32, 2, 128, "q8_0", "q4_0")
    wide = torch.full((2, 9), -1, dtype=torch.int32, device="cuda")
    t = wide[:, 2:8]
    t[0] = torch.tensor([3, 7, 1, 4, 0, 2])
    t[1] = torch.tensor([3, 7, 1, 5, 6, 8])
    k = torch.from_numpy(rng.standard_normal((180, 2, 128)).astype(np.float32)).cuda()
    v = torch.from_numpy(rng.standard_normal((180, 2, 128)).astype(np.float32)).cuda()
    cache.append(k, v, t[:1], dev([180]), cu_q=dev([0, 180]), max_q=180)
    k2, v2 = torch.randn_like(k[:60]), torch.randn_like(v[:60])
    cache.append(k2, v2, t[1:], dev([156]), cu_q=dev([0, 60]), max_q=60)
    q = torch.randn((2 * new, 6, 128), device="cuda").half()
    out = cache.attention(q, t, dev([180, 156]), cu_q=dev([0, new, 2 * new]), max_q=new)
    rows = [(k, v), (torch.cat([k[:96], k2]), torch.cat([v[:96], v2]))]
    for i, (kk, vv) in enumerate(rows):
        ks, vs = torch.from_numpy(stored("q8_0", kk.cpu().numpy())).cuda(), torch.from_numpy(stored("q4_0", vv.cpu().numpy())).cuda()
        o, _, av, qk = attend(q[i * new:(i + 1) * new], ks, vs, 1 / math.sqrt(128))
        tol, _ = bounds(o, av, qk, "f16", 180, 128, True, offset_terms(("q8_0", "q4_0"), q[i * new:(i + 1) * new], ks, vs,
                                                                                     1 / math.sqrt(128), 180))
        assert ((out[i * new:(i + 1) * new].double() - o).abs() <= tol).all()


@pytest.mark.parametrize("new", [1, 33])
def test_captured_steps_follow_the_device(kvq, new):
    """Append + attention captured once and replayed with other lengths, rows and tables; two graphs
    of the same sizes live side by side, an eager call between them."""
    hkv, hq, d, page, width = 2, 8, 128, 16, 20
    cache = kvq.PagedCache(64, page, hkv, d, "q8_0", "q8_0")
    cache.pool.fill_(0xff)
    rng = np.random.default_rng(0)
    rope = kvq.Rope.from_base(width * page, d)
    st = dict(table=torch.zeros((2, width), dtype=torch.int32, device="cuda"), lens=dev([new, new]), cu=dev([0, new, 2 * new]))
    k, v, q = (torch.randn((2 * new, h, d), device="cuda").half() for h in (hkv, hkv, hq))
    st["table"].copy_(torch.from_numpy(rng.permutation(64)[:40].reshape(2, width).astype(np.int32)))

    def step():
        r = cache.append(k, v, st["table"], st["lens"], cu_q=st["cu"], max_q=new, rope=rope, q=q)
        return r, cache.attention(r, st["table"], st["lens"], cu_q=st["cu"], max_q=new)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            graphs.append((g, step()))
    have = [0, 0]
    for i in range(6):
        have = [a + new for a in have]
        st["lens"].copy_(dev(have))
        for x in (k, v, q):
            x.normal_()
        g, (r, out) = graphs[i % 2]
        g.replay()
        got = out.clone()
        eager_r, eager = step()
        assert torch.equal(eager_r, r) and torch.equal(eager, got)
        kk, vv = cache.gather(st["table"], st["lens"], sum(have), cu_q=dev(cumulative(have)), max_q=max(have), dtype=torch.float32)
        for b in range(2):
            at = sum(have[:b])
            o, _, av, qk = attend(r[b * new:(b + 1) * new], kk[at:at + have[b]].double(), vv[at:at + have[b]].double(), 1 / math.sqrt(d))
            tol, _ = bounds(o, av, qk, "f16", have[b], d, True)
            assert ((got[b * new:(b + 1) * new].double() - o).abs() <= tol).all()
    assert cache.read_error() == 0


@pytest.mark.parametrize("new", [1, 48])
def test_streams_at_the_same_time(kvq, new):
    """Reads of one cache on several streams at once give what they give alone, bit for bit."""
    b = Batch(kvq, [3000, 2500], [new, new], hkv=2, pair=("q4_0", "q4_0"), seed=1)
    qs = [b.queries(10, "bf16", seed=s) for s in range(4)]
    alone = [b.cache.attention(q, b.table, b.lens_t, cu_q=b.cu, max_q=new) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    for _ in range(5):
        outs = [b.cache.attention(q, b.table, b.lens_t, cu_q=b.cu, max_q=new, stream=s) for q, s in zip(qs, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(alone, outs))


@pytest.mark.parametrize("new", [1, 8, 60])
def test_own_workspace(kvq, new):
    """A caller's workspace of the reported size holds any garbage before the call and nothing after
    it matters; a smaller one is refused before anything is written."""
    b = Batch(kvq, [700, 90], [new, new], seed=2)
    q = b.queries(4, "f16")
    size = b.cache.workspace_bytes(2, b.n, 4, max_len=b.table.shape[1] * 32, max_q=new, dtype=torch.float16)
    guard = torch.full((size + 256,), 0xff, dtype=torch.uint8, device="cuda")
    out = b.cache.attention(q, b.table, b.lens_t, cu_q=b.cu, max_q=new, workspace=guard[:size])
    b.check(q, "f16", out, None)
    assert bool((guard[size:] == 0xff).all())
    if size > 16:
        keep = torch.full_like(out, 3.0)
        with pytest.raises(kvq.KvqError) as e:
            b.cache.attention(q, b.table, b.lens_t, cu_q=b.cu, max_q=new, workspace=guard[:size - 16], out=keep)
        assert e.value.status == 7 and bool((keep == 3.0).all())


def test_pool_past_four_gigabytes(kvq):
    """Pages whose byte offsets pass 32 bits, at both ends of the pool."""
    page, hkv, d = 256, 8, 128
    per = kvq.paged_size(1, page, hkv, d, "f16", "f16")[0]
    pages = (5 << 30) // per
    cache = kvq.PagedCache(pages, page, hkv, d, "f16", "f16")
    t = dev([[pages - 1, 0, pages // 2 + 1]])
    k = torch.randn((600, hkv, d), device="cuda")
    v = torch.randn((600, hkv, d), device="cuda")
    cache.append(k, v, t, dev([600]), cu_q=dev([0, 600]), max_q=600)
    gk, gv = cache.gather(t, dev([600]), 600, cu_q=dev([0, 600]), max_q=600)
    assert torch.equal(gk, k.half()) and torch.equal(gv, v.half())
    for new in (1, 40):
        q = torch.randn((new, 16, d), device="cuda").bfloat16()
        out = cache.attention(q, t, dev([600]), cu_q=dev([0, new]), max_q=new)
        o, _, av, qk = attend(q, k.half().double(), v.half().double(), 1 / math.sqrt(d))
        tol, _ = bounds(o, av, qk, "bf16", 600, d, True)
        assert ((out.double() - o).abs() <= tol).all()


@pytest.mark.parametrize("pair", [("q8_0", "q4_0"), ("q4_0", "q4_0")])
def test_prompt_then_tokens_as_the_contiguous_cache(kvq, pair):
    """A serving run: a prompt in two chunks, then single tokens, through append and attention; the
    contiguous cache with the same rows agrees (both within their bounds of the same attention)."""
    hkv, hq, d, page = 2, 10, 128, 32
    rope = kvq.Rope.from_base(400, d)
    cache = kvq.PagedCache(16, page, hkv, d, *pair)
    flat = kvq.KVCache(1, hkv, d, 400, *pair)
    t = dev([np.random.default_rng(1).permutation(16)[:13]])
    at = 0
    for n in [150, 90] + [1] * 12:
        at += n
        k, v, q = (torch.randn((n, h, d), device="cuda") for h in (hkv, hkv, hq))
        args = dict(cu_q=dev([0, n]), max_q=n)
        r = cache.append(k, v, t, dev([at]), rope=rope, q=q, **args)
        out, lse = cache.attention(r[-1:].contiguous(), t, dev([at]), return_lse=True)
        # the contiguous cache takes rotated rows: read them back unquantised through an f16 twin
        kr = torch.from_numpy(rotate(k.cpu().numpy(), rope.cos_sin.cpu().numpy(), np.arange(at - n, at), d, False)).cuda()
        flat.append(kr.permute(1, 0, 2)[None].contiguous(), v.permute(1, 0, 2)[None].contiguous())
        ref, ref_lse = flat.decode(r[-1:].contiguous())
        kk, vv = cache.gather(t, dev([at]), at, cu_q=dev([0, at]), max_q=at, dtype=torch.float32)
        o, z, av, qk = attend(r[-1:], kk.double(), vv.double(), 1 / math.sqrt(d))
        tol, ltol = bounds(o, av, qk, "f32", at, d, False, offset_terms(pair, r[-1:], kk, vv, 1 / math.sqrt(d), at))
        assert ((out.double() - o).abs() <= tol).all() and ((lse.double() - z).abs() <= ltol).all()
        assert ((ref.double() - out.double()).abs() <= 2 * tol).all()
        chunk = cache.attention(r.bfloat16(), t, dev([at]), **args)
        o, _, av, qk = attend(r.bfloat16(), kk.double(), vv.double(), 1 / math.sqrt(d))
        tol, _ = bounds(o, av, qk, "bf16", at, d, True, offset_terms(pair, r, kk, vv, 1 / math.sqrt(d), at))
        assert ((chunk.double() - o).abs() <= tol).all()
    assert cache.read_error() == 0
