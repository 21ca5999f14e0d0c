"""Operators of the paged quantised KV cache: the cases that are measured, their plain form in
elementary torch operations, and the calls a program makes of the framework.

Three operators share one cache format and one description of a batch (block table, lengths,
query offsets):

  append     rotate keys (and queries) by their positions, quantise the rows into their pages
  gather     read rows of the cache back as values
  attention  causal grouped-query attention of each sequence's new tokens over its pages
"""
import math

import numpy as np
import torch

own = False

BLOCK = 32  # values per quantisation block
ROPE_BASE = 1000000.0
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
ROW_BYTES = {"f16": 2.0, "q8_0": 34 / 32, "q4_0": 18 / 32}  # stored bytes per value
PAIRS = [("f16", "f16"), ("q8_0", "q8_0"), ("q8_0", "q4_0"), ("q4_0", "q4_0")]


def _case(name, op, kv, q, dim, tk, tv, dtype, page, seqs, len_min, len_max, new_min=1, new_max=1, rot=0,
          interleaved=False):
    return {"name": name, "op": op, "heads_kv": kv, "heads_q": q, "dim": dim, "type_k": tk, "type_v": tv,
            "dtype": dtype, "page": page, "seqs": seqs, "len_min": len_min, "len_max": len_max, "new_min": new_min,
            "new_max": new_max, "rot": rot, "interleaved": interleaved}


def listed():
    # shapes: the dense model (8 KV heads, 40 query heads, D 128) and the hybrid one (2, 16, 256)
    return [
        # one new token of one sequence: the latency of a decode step's write
        _case("append_token", "append", 8, 40, 128, "q8_0", "q8_0", "bf16", 16, 1, 8193, 8193, 1, 1, 128),
        # a decode step of a serving batch: one token each, anywhere in their pages
        _case("append_batch", "append", 8, 40, 128, "q8_0", "q4_0", "f16", 64, 64, 17, 16384, 1, 1, 128),
        # prompts of three sequences, short to long, starting inside pages and tiles
        _case("append_chunk", "append", 8, 40, 128, "q4_0", "q4_0", "bf16", 128, 3, 1000, 9001, 333, 8192, 128),
        # wide heads with a partial, interleaved rotation and 32-bit activations
        _case("append_hybrid", "append", 2, 16, 256, "q8_0", "q8_0", "f32", 32, 2, 4096, 5001, 2047, 2049, 64, True),
        # short sequences read back whole
        _case("gather_short", "gather", 8, 40, 128, "q4_0", "q4_0", "f16", 16, 5, 1, 777),
        # a long sequence exported, 16-bit values
        _case("gather_long", "gather", 8, 40, 128, "q8_0", "q4_0", "bf16", 64, 1, 65536, 65536),
        # one token over a short context: launch latency
        _case("decode_short", "attention", 8, 40, 128, "q4_0", "q4_0", "bf16", 16, 1, 513, 513),
        # one token over a very long context in 4 bits
        _case("decode_long", "attention", 8, 40, 128, "q4_0", "q4_0", "bf16", 64, 1, 131072, 131072),
        # a decode step of 16 sequences of 8K to 64K, the default asymmetric tier
        _case("decode_batch", "attention", 8, 40, 128, "q8_0", "q4_0", "f16", 64, 16, 8192, 65536),
        # wide heads, odd lengths, 32-bit activations
        _case("decode_hybrid", "attention", 2, 16, 256, "q8_0", "q8_0", "f32", 256, 4, 4095, 65535),
        # the last chunk of a long prompt
        _case("prefill", "attention", 8, 40, 128, "q4_0", "q4_0", "bf16", 64, 1, 16384, 16384, 4096, 4096),
        # a mixed step: chunks of several sequences and single tokens beside them
        _case("extend_hybrid", "attention", 2, 16, 256, "q8_0", "q8_0", "f16", 32, 6, 100, 16001, 1, 700),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["append", "gather", "attention", "attention", "attention"])
    dim = rng.choice([128, 128, 256])
    kv = rng.choice([1, 2, 4, 8])
    q = kv * rng.choice([1, 2, 4, 5, 7, 8, 16])
    tk, tv = rng.choice(PAIRS)
    page = rng.choice([16, 32, 48, 64, 128, 256])
    dtype = rng.choice(["bf16", "f16", "f32"])
    if op == "append":
        seqs = _log(rng, 1, 64)
        new = _log(rng, 1, max(1, 8192 // seqs))
        top = _log(rng, max(new, 16), 32768)
        return _case("", op, kv, q, dim, tk, tv, dtype, page, seqs, rng.randint(1, top), top, rng.randint(1, new), new,
                     rng.choice([0, dim, dim, 64, 96]), rng.random() < 0.3)
    if op == "gather":
        seqs = _log(rng, 1, 32)
        top = _log(rng, 1, 65536 // seqs)
        return _case("", op, kv, q, dim, tk, tv, dtype, page, seqs, rng.randint(1, top), top)
    if rng.random() < 0.5:  # one token per sequence
        seqs = _log(rng, 1, 64)
        top = _log(rng, 1, min(131072, (1 << 20) // seqs * 128 // dim))
        return _case("", op, kv, q, dim, tk, tv, dtype, page, seqs, rng.randint(1, top), top)
    seqs = _log(rng, 1, 8)
    top = _log(rng, 32, 16384)
    most = 16 if dtype == "f32" else 4096
    # at most half the query-head work of the longest chunk listed
    new = min(top, _log(rng, 2, max(2, min(most, 4096 * 40 * 64 // (q * dim // 2 * seqs)))))
    return _case("", op, kv, q, dim, tk, tv, dtype, page, seqs, rng.randint(1, top), top, rng.randint(1, new), new)


def _spread(lo, hi, n):
    """n sizes between lo and hi, even over the logarithm."""
    return [hi] if n == 1 else [round(lo * (hi / lo) ** (i / (n - 1))) for i in range(n)]


def _sizes(case):
    """(lengths, new tokens) of the sequences; the lengths include the new tokens."""
    n = case["seqs"]
    lens = _spread(case["len_min"], case["len_max"], n)
    if case["op"] == "gather":
        return lens, lens
    new = _spread(case["new_min"], case["new_max"], n)
    return lens, [min(a, b) for a, b in zip(new, lens)]


def work(case):
    lens, new = _sizes(case)
    kv, hq, d = case["heads_kv"], case["heads_q"], case["dim"]
    row = kv * d * (ROW_BYTES[case["type_k"]] + ROW_BYTES[case["type_v"]])
    n, e = sum(new), BYTES[case["dtype"]]
    if case["op"] == "append":
        # keys, values and queries in, rows and queries out, one row of angles per token
        return {"bytes": n * (2 * kv * d * e + 2 * hq * d * e + row + 4 * case["rot"]), "flops": n * (kv + hq) * case["rot"] * 3}
    if case["op"] == "gather":
        return {"bytes": n * (row + 2 * kv * d * e), "flops": 2 * n * kv * d}
    pairs = sum(m * a - m * (m - 1) // 2 for a, m in zip(lens, new))
    return {"bytes": sum(lens) * row + 2 * n * hq * d * e, "flops": 4 * pairs * hq * d}


def _rows(seed, count, heads, dim, outliers):
    """Normal rows; keys have four outlier channels per head, ten times as large."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((count, heads, dim), generator=g, device="cuda")
    if outliers:
        at = torch.rand((heads, dim), generator=g, device="cuda").argsort(-1)[:, :4]
        x *= torch.ones((heads, dim), device="cuda").scatter_(1, at, 10.0)
    return x


def _angles(count, rot):
    """[count, rot] float32: cosines, then sines of position * base^(-2j / rot), the angles in 64 bits."""
    j = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    a = torch.arange(count, dtype=torch.float64, device="cuda")[:, None] * ROPE_BASE ** (-2.0 * j / max(rot, 1))
    return torch.cat([a.cos(), a.sin()], -1).float().contiguous()


def _inputs(case, seed):
    """Tensors both forms and the 64-bit definition start from."""
    lens, new = _sizes(case)
    kv, hq, d, page = case["heads_kv"], case["heads_q"], case["dim"], case["page"]
    dtype = DTYPES[case["dtype"]]
    n, width = sum(new), -(-max(lens) // page)
    need = [-(-a // page) for a in lens]
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    pages = sum(need) + 3
    perm = torch.randperm(pages, generator=g, device="cuda").int()
    table = np.zeros((len(lens), width), np.int64)
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = np.arange(at, at + k)
        at += k
    s = {"case": case, "pages": pages, "n": n, "max_q": max(new), "max_len": max(lens)}
    s["table"] = perm[torch.from_numpy(table).cuda()].contiguous()
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["cu_q"] = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32, device="cuda")
    if case["op"] == "append":
        s["k"] = _rows(seed + 2, n, kv, d, True).to(dtype)
        s["v"] = _rows(seed + 3, n, kv, d, False).to(dtype)
        s["angles"] = _angles(max(lens), case["rot"]) if case["rot"] else None
    else:  # what the cache holds: every row of every sequence
        total = sum(lens)
        s["k_rows"] = _rows(seed + 2, total, kv, d, True)
        s["v_rows"] = _rows(seed + 3, total, kv, d, False)
        s["cu_rows"] = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device="cuda")
    if case["op"] != "gather":
        s["q"] = _rows(seed + 4, n, hq, d, False).to(dtype)
    return s


def _where(table, lens, cu, page):
    """(sequence, position, cache row) of every packed token."""
    t = torch.arange(int(cu[-1]), device="cuda")
    b = torch.searchsorted(cu[1:].long(), t, right=True)
    p = lens[b].long() - (cu[b + 1].long() - t)
    return b, p, table[b, p // page].long() * page + p % page


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        # the handle that a program keeps, with what its earlier steps wrote
        import quantised_kv_long_gb300 as kvq
        cache = kvq.PagedCache(s["pages"], case["page"], case["heads_kv"], case["dim"], case["type_k"], case["type_v"])
        s["cache"] = cache
        if case["op"] == "append":
            s["rope"] = kvq.Rope(s["angles"], interleaved=case["interleaved"]) if case["rot"] else None
        else:
            cache.append(s.pop("k_rows"), s.pop("v_rows"), s["table"], s["lens"], cu_q=s.pop("cu_rows"), max_q=s["max_len"])
    else:
        rows = s["pages"] * case["page"]
        s["store_k"] = _store(case["type_k"], rows, case["heads_kv"], case["dim"])
        s["store_v"] = _store(case["type_v"], rows, case["heads_kv"], case["dim"])
        if case["op"] != "append":
            _, _, at = _where(s["table"], s["lens"], s.pop("cu_rows"), case["page"])
            _put(s["store_k"], case["type_k"], at, s.pop("k_rows"))
            _put(s["store_v"], case["type_v"], at, s.pop("v_rows"))
    if case["op"] == "attention":
        s["b"], s["p"], _ = _where(s["table"], s["lens"], s["cu_q"], case["page"])
    elif not own:
        s["b"], s["p"], s["at"] = _where(s["table"], s["lens"], s["cu_q"], case["page"])
    return s


def run(s):
    case = s["case"]
    if own:
        cache, where = s["cache"], dict(cu_q=s["cu_q"], max_q=s["max_q"])
        if case["op"] == "append":
            q = cache.append(s["k"], s["v"], s["table"], s["lens"], rope=s["rope"], q=s["q"], **where)
            k, v = cache.gather(s["table"], s["lens"], s["n"], dtype=torch.float16, **where)
            return {"q": q, "k": k, "v": v}
        if case["op"] == "gather":
            k, v = cache.gather(s["table"], s["lens"], s["n"], dtype=DTYPES[case["dtype"]], **where)
            return {"k": k, "v": v}
        if s["max_q"] == 1:
            out, lse = cache.attention(s["q"], s["table"], s["lens"], max_len=s["max_len"], return_lse=True)
            return {"out": out, "lse": lse}
        return {"out": cache.attention(s["q"], s["table"], s["lens"], max_len=s["max_len"], **where)}
    if case["op"] == "append":
        k, q = s["k"].float(), s["q"].float()
        if case["rot"]:
            k = _rotate(k, s["angles"][s["p"]], case["rot"], case["interleaved"])
            q = _rotate(q, s["angles"][s["p"]], case["rot"], case["interleaved"])
        _put(s["store_k"], case["type_k"], s["at"], k)
        _put(s["store_v"], case["type_v"], s["at"], s["v"].float())
        return {"q": q.to(s["q"].dtype), "k": _get(s["store_k"], case["type_k"], s["at"]).half(),
                "v": _get(s["store_v"], case["type_v"], s["at"]).half()}
    if case["op"] == "gather":
        dtype = DTYPES[case["dtype"]]
        return {"k": _get(s["store_k"], case["type_k"], s["at"]).to(dtype), "v": _get(s["store_v"], case["type_v"], s["at"]).to(dtype)}
    out, lse = _attend(s)
    return {"out": out, "lse": lse} if s["max_q"] == 1 else {"out": out}


# ---- the plain form ----

def _store(kind, rows, heads, dim):
    if kind == "f16":
        return [torch.zeros((rows, heads, dim), dtype=torch.float16, device="cuda")]
    codes = torch.zeros((rows, heads, dim), dtype=torch.int8, device="cuda")
    return [codes, torch.zeros((rows, heads, dim // BLOCK), dtype=torch.float16, device="cuda")]


def _put(store, kind, at, x):
    """Quantise float32 rows [n, heads, dim] into rows `at` of the store."""
    if kind == "f16":
        store[0][at] = x.half()
        return
    x = x.unflatten(-1, (-1, BLOCK))
    if kind == "q8_0":
        top = x.abs().amax(-1, keepdim=True)
        d = top / torch.full_like(top, 127.0)
        y = x * torch.where(d != 0, torch.ones_like(d) / d, torch.zeros_like(d))
        t = y.trunc()
        c = t + torch.where((y - t).abs() >= 0.5, y.sign(), torch.zeros_like(y))
    else:
        d = x.gather(-1, x.abs().argmax(-1, keepdim=True)) / torch.full_like(x[..., :1], -8.0)
        y = x * torch.where(d != 0, torch.ones_like(d) / d, torch.zeros_like(d))
        c = (y + 8.5).trunc().clamp(max=15.0) - 8.0
    store[0][at] = c.to(torch.int8).flatten(-2)
    store[1][at] = d.half()[..., 0]


def _get(store, kind, at):
    """float32 values of rows `at` (any shape of indices)."""
    if kind == "f16":
        return store[0][at].float()
    return (store[0][at].unflatten(-1, (-1, BLOCK)).float() * store[1][at].float()[..., None]).flatten(-2)


def _rotate(x, angles, rot, interleaved):
    c, s = angles[:, None, :rot // 2], angles[:, None, rot // 2:]
    head, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        a, b = head[..., 0::2], head[..., 1::2]
        turned = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    else:
        a, b = head[..., :rot // 2], head[..., rot // 2:]
        turned = torch.cat([a * c - b * s, b * c + a * s], -1)
    return torch.cat([turned, rest], -1)


def _attend(s):
    case, seqs = s["case"], s["case"]["seqs"]
    kv, hq, d, page, top = case["heads_kv"], case["heads_q"], case["dim"], case["page"], s["max_len"]
    pos = torch.arange(top, device="cuda")
    # rows past a sequence's length point at some page and are masked
    at = s["table"][:, pos // page].long() * page + pos % page
    k = _get(s["store_k"], case["type_k"], at).permute(0, 2, 3, 1)  # [seqs, kv, d, top]
    v = _get(s["store_v"], case["type_v"], at).permute(0, 2, 1, 3)  # [seqs, kv, top, d]
    # queries padded to [seqs, max_q]
    i = torch.arange(s["n"], device="cuda") - s["cu_q"][s["b"]].long()
    q = torch.zeros((seqs, s["max_q"], hq, d), device="cuda")
    q[s["b"], i] = s["q"].float()
    last = torch.full((seqs, s["max_q"]), -1, device="cuda", dtype=torch.long)
    last[s["b"], i] = s["p"]
    q = q.unflatten(2, (kv, hq // kv)).permute(0, 2, 3, 1, 4).flatten(2, 3)  # [seqs, kv, G max_q, d]
    w = (q @ k).mul_(1.0 / math.sqrt(d)).unflatten(2, (hq // kv, s["max_q"]))
    seen = pos <= last[:, None, None, :, None]
    w.masked_fill_(~seen, -math.inf)
    m = w.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    w.sub_(m).exp_()
    l = w.sum(-1, keepdim=True)
    o = (w.flatten(2, 3) @ v).unflatten(2, (hq // kv, s["max_q"])) / torch.where(l > 0, l, torch.ones_like(l))
    lse = (m + l.log())[..., 0]
    o = o.permute(0, 3, 1, 2, 4).flatten(2, 3)[s["b"], i]
    return o.to(s["q"].dtype), lse.permute(0, 3, 1, 2).flatten(2, 3)[s["b"], i]


# ---- the definition in 64 bits ----

def _round_f16(x):
    return x.to(torch.float16).double()


def _values(kind, x):
    """What rows of a type stand for, in float64.  The quantiser is defined on float32 values with one
    rounding per operation, its scale as float16: its codes are whole numbers, so nothing else will do."""
    if kind == "f16":
        return _round_f16(x)
    shape = x.shape
    x = x.reshape(-1, BLOCK).float()
    big, at = x.abs().max(-1, keepdim=True)
    # quotients of float32 values, rounded once: the float64 quotient is within 2^-53 of the true one
    if kind == "q8_0":
        step = (big.double() / 127.0).float()
    else:
        step = torch.gather(x, 1, at) / -8.0
    inverse = torch.where(step != 0, (1.0 / step.double()).float(), torch.zeros_like(step))
    y = (x.double() * inverse.double()).float()
    if kind == "q8_0":
        code = torch.floor(y.abs().double() + 0.5) * y.sign()
    else:
        code = torch.floor((y.double() + 8.5).float()).clamp(max=15.0).double() - 8.0
    return (code * _round_f16(step.double())).reshape(shape)


def exact(case, seed):
    s = _inputs(case, seed)
    lens, new = _sizes(case)
    if case["op"] == "append":
        pos = torch.cat([torch.arange(a - m, a, device="cuda") for a, m in zip(lens, new)])
        turned = []
        for x in (s["k"].double(), s["q"].double()):
            r = case["rot"]
            if r:
                ang = s["angles"].double()[pos]
                z = torch.polar(torch.ones_like(ang[:, :r // 2]), torch.zeros_like(ang[:, :r // 2]))
                z = z * torch.complex(ang[:, :r // 2], ang[:, r // 2:])
                head = x[..., :r]
                w = torch.complex(head[..., 0::2], head[..., 1::2]) if case["interleaved"] else torch.complex(head[..., :r // 2], head[..., r // 2:])
                w = w * z[:, None]
                x = x.clone()
                if case["interleaved"]:
                    x[..., 0:r:2], x[..., 1:r:2] = w.real, w.imag
                else:
                    x[..., :r // 2], x[..., r // 2:r] = w.real, w.imag
            turned.append(x)
        return {"q": turned[1], "k": _values(case["type_k"], turned[0]), "v": _values(case["type_v"], s["v"].double())}
    if case["op"] == "gather":
        return {"k": _values(case["type_k"], s["k_rows"].double()), "v": _values(case["type_v"], s["v_rows"].double())}
    kv, hq, d = case["heads_kv"], case["heads_q"], case["dim"]
    group = hq // kv
    out = torch.zeros((s["n"], hq, d), dtype=torch.float64, device="cuda")
    lse = torch.zeros((s["n"], hq), dtype=torch.float64, device="cuda")
    row, tok = 0, 0
    for a, m in zip(lens, new):
        for h in range(kv):
            k = _values(case["type_k"], s["k_rows"][row:row + a, h].double())
            v = _values(case["type_v"], s["v_rows"][row:row + a, h].double())
            for t in range(0, m, 512):
                n = min(512, m - t)
                end = a - m + t + n  # keys that the last query of the piece sees
                q = s["q"][tok + t:tok + t + n, h * group:(h + 1) * group].double()
                w = torch.einsum("tgd,kd->tgk", q, k[:end]) / math.sqrt(d)
                hide = torch.arange(end, device="cuda")[None] > (torch.arange(n, device="cuda") + a - m + t)[:, None]
                w.masked_fill_(hide[:, None], -math.inf)
                z = torch.logsumexp(w, -1)
                out[tok + t:tok + t + n, h * group:(h + 1) * group] = torch.einsum("tgk,kd->tgd", (w - z[..., None]).exp(), v[:end])
                lse[tok + t:tok + t + n, h * group:(h + 1) * group] = z
        row, tok = row + a, tok + m
    return {"out": out, "lse": lse} if max(new) == 1 else {"out": out}
