"""Cases of the low-precision serving path: the 8-bit linear layer, the 4-bit paged cache and the attention over it.

A serving step of one layer reads its weights, its users' cached keys and values and little else, so what these three
save is bytes: the projections multiply 8-bit integers (one scale a token, one a channel), the cache holds four bits an
element (one scale and one zero point for each token and head), and the attention reads that cache as it is.

`run` computes an operator in its plain form (elementary torch operations in 32 bits, 64 where a value decides between
two codes or two time buckets) or, with `own`, by the library's entry points.  `exact` is the definition in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
DEV = "cuda"
N_BUCKETS = 128
EPS = 1e-5
TINY = 2.0 ** -126  # a scale below the smallest normal number: the row counts as zeros


# ---------------------------------------------------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------------------------------------------------
def _linear(name, t, k, n, x, out, silu, bias):
    return {"name": name, "op": "linear", "T": t, "K": k, "N": n, "x": x, "out": out, "silu": silu, "bias": bias}


def _append(name, b, lo, hi, cached, h, d, page, dtype):
    return {"name": name, "op": "append", "B": b, "new_lo": lo, "new_hi": hi, "cached": cached, "H": h, "d": d,
            "page": page, "dtype": dtype}


def _attn(name, b, rlo, rhi, cand, clo, chi, h, d, page, dtype, n_max):
    return {"name": name, "op": "attn", "B": b, "rows_lo": rlo, "rows_hi": rhi, "cand": cand, "cached_lo": clo,
            "cached_hi": chi, "H": h, "d": d, "page": page, "dtype": dtype, "n_max": n_max}


def listed():
    return [
        # one new action of each of 8 users through a layer's input projection: latency
        _linear("i8 f1, 8 rows", 8, 512, 2048, "bf16", "bf16", True, True),
        # the output projection of a request of 8 users with 128 new tokens each
        _linear("i8 f2, 1024 rows", 1024, 512, 512, "bf16", "bf16", False, True),
        # the input projection of a whole batch of long users (a cold start: everything is computed)
        _linear("i8 f1, 53095 rows", 53095, 512, 2048, "bf16", "bf16", True, True),
        # a wide model's projection with odd sizes and 32-bit results (a scoring head)
        _linear("i8 wide, odd, 32 bits", 1537, 2064, 5000, "f32", "f32", False, False),
        # every user's newest action goes into the cache and is read back: latency
        _append("q4 append, 64 x 1", 64, 1, 1, 1000, 4, 128, 32, "bf16"),
        # a request's 64 new actions of 8 users
        _append("q4 append, 8 x 64", 8, 64, 64, 6000, 4, 128, 32, "bf16"),
        # the histories of 32 new users of 512 to 1024 tokens are cached at once
        _append("q4 append, 32 x 512..1024", 32, 512, 1024, 0, 4, 128, 32, "bf16"),
        # one user with a short history and one new action: latency
        _attn("q4 attn, 1 user, 1 row", 1, 1, 1, 0, 100, 100, 4, 128, 32, "bf16", 1024),
        # one new action of each of 64 users against their whole histories
        _attn("q4 attn, 64 users, 1 row", 64, 1, 1, 0, 1000, 8192, 4, 128, 32, "bf16", 8320),
        # a request of 8 users: 64 new actions and 64 candidates each
        _attn("q4 attn, 8 users, 128 rows", 8, 128, 128, 64, 6144, 8192, 4, 128, 32, "bf16", 8320),
        # ranking: 512 candidates of each of 16 users against the cached history
        _attn("q4 attn, 16 users, 512 cand", 16, 512, 512, 512, 2048, 4096, 4, 128, 32, "bf16", 4608),
        # a small model in 32 bits with odd heads, pages and lengths
        _attn("q4 attn, odd, 32 bits", 5, 0, 37, 7, 0, 900, 3, 64, 24, "f32", 1024),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "append", "attn"])
    if op == "linear":
        while True:
            t, k, n = _log(rng, 1, 60000), 16 * _log(rng, 4, 256), 8 * _log(rng, 8, 1024)
            if t * k * n <= 53095 * 512 * 2048 and t * n <= 53095 * 2048:
                break
        c = _linear("", t, k, n, rng.choice(["bf16", "bf16", "f32"]), rng.choice(["bf16", "bf16", "f32"]),
                    rng.random() < 0.5, rng.random() < 0.7)
    elif op == "append":
        while True:
            b, hi = _log(rng, 1, 100), _log(rng, 1, 1024)
            h, d = rng.choice([1, 2, 3, 4, 8]), rng.choice([32, 64, 96, 128])
            if b * hi * h * d <= 32 * 1024 * 512:
                break
        c = _append("", b, rng.choice([0, 1, hi]) if hi > 1 else 1, hi, rng.choice([0, 1, 31, _log(rng, 1, 4000)]), h, d,
                    rng.choice([8, 16, 24, 32, 64, 128]), rng.choice(["bf16", "bf16", "f32"]))
    else:
        while True:
            b, rows = _log(rng, 1, 64), _log(rng, 1, 512)
            chi = _log(rng, 16, 8192)
            f32 = rng.random() < 0.25
            h, d = rng.choice([(4, 128), (2, 128), (8, 128), (1, 128), (3, 64), (4, 32)])
            cost = b * rows * (chi + rows) * h * d
            if cost <= 16 * 512 * 4608 * 512 // (16 if f32 or d != 128 else 1) and b * chi * h * d <= 64 * 8192 * 512:
                break
        c = _attn("", b, rng.choice([0, rows, max(1, rows // 2)]), rows, rng.choice([0, rows // 2, rows]),
                  rng.choice([0, chi // 3, chi]), chi, h, d, rng.choice([8, 16, 24, 32, 64, 128]),
                  "f32" if f32 else "bf16", chi + rows + rng.choice([0, 1, 128]))
        if c["rows_lo"] == 0 and b == 1:
            c["rows_lo"] = rows
    del c["name"]
    return c


def _lengths(c):
    """The users' lengths of a case: the same for every seed, both ends of each range among them."""
    r = random.Random("lengths %d %d" % (c["B"], c.get("new_hi", c.get("rows_hi"))))

    def some(lo, hi):
        v = [r.randint(lo, hi) for _ in range(c["B"])]
        v[-1] = hi
        if c["B"] > 1:
            v[0] = lo
        return v

    if c["op"] == "append":
        new = some(c["new_lo"], c["new_hi"])
        return new, [max(0, c["cached"] - 3 * (u % 5)) for u in range(c["B"])]
    rows = some(c["rows_lo"], c["rows_hi"])
    cached = some(c["cached_lo"], c["cached_hi"])
    return rows, cached


def work(c):
    """One pass: each input read once, each output written once, the products' operations."""
    if c["op"] == "linear":
        t, k, n = c["T"], c["K"], c["N"]
        by = t * k * (2 if c["x"] == "bf16" else 4) + n * k + t * n * (2 if c["out"] == "bf16" else 4) + 8 * n
        return {"bytes": by, "flops": 2 * t * k * n}
    es = 2 if c["dtype"] == "bf16" else 4
    h, d = c["H"], c["d"]
    row4 = h * (d // 2 + 4)  # a token's keys (or values) in the cache
    if c["op"] == "append":
        new, _ = _lengths(c)
        return {"bytes": sum(new) * 2 * (h * d * es + row4 + row4 + h * d * es), "flops": sum(new) * 2 * h * d * 6}
    rows, cached = _lengths(c)
    by = fl = 0
    for r, l in zip(rows, cached):
        cand = min(c["cand"], r)
        hist = r - cand
        pairs = hist * l + hist * (hist + 1) // 2 + cand * (l + hist + 1)
        by += (l * 2 * row4 + (l + r) * 8 if r else 0) + r * h * d * es * 5
        fl += pairs * h * d * 4
    return {"bytes": by, "flops": fl}


# ---------------------------------------------------------------------------------------------------------------------
# the 4-bit form of a row: v = scale * (code - zero)
# ---------------------------------------------------------------------------------------------------------------------
def _quant4(x):
    """[..., d] 32-bit rows -> codes 0..15 (uint8), scale and zero point (bf16), each row by itself."""
    lo = x.amin(-1).clamp(max=0.0)
    hi = x.amax(-1).clamp(min=0.0)
    s = ((hi - lo) / torch.full_like(hi, 15.0)).bfloat16().float()
    use = torch.where(s >= TINY, s, torch.ones_like(s)).double()
    zero = (-lo.double() / use).round().clamp(0, 15)
    code = ((x.double() / use[..., None]).round() + zero[..., None]).clamp(0, 15)
    live = s >= TINY
    code = torch.where(live[..., None], code, torch.zeros_like(code)).to(torch.uint8)
    return code, torch.where(live, s, torch.zeros_like(s)).bfloat16(), torch.where(live, zero, torch.zeros_like(zero)).bfloat16()


def _pack4(code):
    """Codes [..., d] -> bytes [..., d / 2]: in each group of 8 elements (4 bytes) nibble i holds element 2 i and
    nibble i + 4 element 2 i + 1 (nibble 0 is the low half of byte 0)."""
    n = code.unflatten(-1, (-1, 4, 2)).transpose(-1, -2).flatten(-2)  # the group's nibbles in order
    n = n.unflatten(-1, (4, 2))
    return (n[..., 0] | (n[..., 1] << 4)).flatten(-2)


def _unpack4(byte):
    n = torch.stack([byte & 15, byte >> 4], -1).flatten(-2).unflatten(-1, (-1, 2, 4))
    return n.transpose(-1, -2).flatten(-3)


def _dequant4(byte, meta):
    """Pool bytes [..., d / 2] and their (scale, zero) [..., 2] -> 32-bit rows [..., d]."""
    m = meta.float()
    return m[..., :1] * (_unpack4(byte).float() - m[..., 1:])


# ---------------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------------
def _silu(x):
    return x / (1 + torch.exp(-x))


def _offsets(v):
    return torch.tensor([0] + list(np.cumsum(v)), dtype=torch.int32, device=DEV)


def _rand(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _table(g, lens, spare, page, h, d):
    """A page table for users of `lens` tokens with room for `spare` more each, pages in random order."""
    have = [-(-l // page) for l in lens]
    need = [-(-(l + s) // page) - a for l, s, a in zip(lens, spare, have)]
    pages = sum(have) + sum(need) + 3
    width = max(1, max(a + b for a, b in zip(have, need)))
    perm = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    rows = torch.full((len(lens), width), -1, dtype=torch.int32)
    at, host = 0, perm.cpu()
    for u, n in enumerate(have):
        rows[u, :n] = host[at:at + n]
        at += n
    free = torch.full((pages,), -1, dtype=torch.int32, device=DEV)
    free[:pages - at] = perm[at:]
    return rows.to(DEV), free, pages - at, pages


def _pool(g, pages, page, h, d, table, lens):
    """A cache of SiLU-activated rows; slots that hold no token are left unusable (their scale is not a number)."""
    k, m = [], []
    step = max(1, (1 << 26) // (h * page * d))
    for p0 in range(0, pages, step):
        code, s, z = _quant4(_silu(_rand(g, min(step, pages - p0), h, page, d) * 1.5))
        k.append(_pack4(code))
        m.append(torch.stack([s, z], -1))
    byte, meta = torch.cat(k), torch.cat(m)
    live = torch.zeros(pages, page, dtype=torch.bool, device=DEV)
    x = torch.arange(table.shape[1], device=DEV)[None, :, None] * page + torch.arange(page, device=DEV)
    held = x < torch.tensor(lens, device=DEV)[:, None, None]
    live[table.clamp(min=0)[:, :, None].expand_as(held)[held].long(), (x % page).expand_as(held)[held]] = True
    meta = torch.where(live[:, None, :, None], meta, torch.full_like(meta, float("nan")))
    byte = torch.where(live[:, None, :, None], byte, torch.full_like(byte, 255))
    return byte.contiguous(), meta.contiguous()


def prepare(c, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 7919 + 17)
    if c["op"] == "linear":
        t, k, n = c["T"], c["K"], c["N"]
        # a layer's input or gated output: tokens of different size
        x = (_rand(g, t, k) * torch.exp(0.5 * _rand(g, t, 1))).to(DT[c["x"]])
        w = (_rand(g, n, k) * math.sqrt(2.0 / (k + n))).bfloat16().float()  # channel by channel
        amax = w.abs().amax(1)
        scale = amax / torch.full_like(amax, 127.0)
        wq = (w.double() / scale.double()[:, None]).round().clamp(-127, 127).to(torch.int8)
        return {"c": c, "x": x, "w_q": wq, "w_scale": scale, "bias": 0.1 * _rand(g, n) if c["bias"] else None}
    h, d, page, dt = c["H"], c["d"], c["page"], DT[c["dtype"]]
    if c["op"] == "append":
        new, cached = _lengths(c)
        table, free, count, pages = _table(g, cached, new, page, h, d)
        total = sum(new)
        # one buffer for what an append changes, so that it can be put back with one copy
        b, w = table.shape
        ints = torch.cat([table.flatten(), torch.tensor(cached, dtype=torch.int32, device=DEV),
                          torch.tensor([count], dtype=torch.int32, device=DEV)])
        live = ints.clone()
        st = {"c": c, "ints": ints, "live": live, "table": live[:b * w].view(b, w), "lens": live[b * w:b * w + b],
              "count": live[b * w + b:], "free": free, "pages": pages, "offsets": _offsets(new), "total": total,
              "starts": torch.tensor(cached, dtype=torch.int32, device=DEV), "most": max(new),
              "k": _silu(_rand(g, total, h, d) * 1.5).to(dt), "v": _silu(_rand(g, total, h, d) * 1.5).to(dt)}
        for x in ("k", "v"):
            st[x + "_pool"] = torch.zeros(pages, h, page, d // 2, dtype=torch.uint8, device=DEV)
            st[x + "_meta"] = torch.zeros(pages, h, page, 2, dtype=torch.bfloat16, device=DEV)
        return st
    rows, cached = _lengths(c)
    table, _, _, pages = _table(g, cached, [0] * c["B"], page, h, d)
    total = sum(rows)
    st = {"c": c, "offsets": _offsets(rows), "lens": torch.tensor(cached, dtype=torch.int32, device=DEV), "table": table,
          "cand": torch.tensor([min(c["cand"], r) for r in rows], dtype=torch.int32, device=DEV) if c["cand"] else None,
          "rows": rows, "cached": cached, "total": total, "max_rows": max(rows), "max_cached": max(cached)}
    for x in ("k", "v"):
        st[x + "_pool"], st[x + "_meta"] = _pool(g, pages, page, h, d, table, cached)
    # one projection's output holds the four blocks side by side, as the layer's f1 writes it
    f1 = _silu(_rand(g, total, 4 * h * d) * 1.5).to(dt)
    hd = h * d
    st["u"] = f1[:, :hd]
    st["v"], st["q"], st["k"] = (f1[:, i * hd:(i + 1) * hd].unflatten(1, (h, d)) for i in (1, 2, 3))
    # seconds between actions are exponential; candidates carry the time of the last action
    n = [a + b for a, b in zip(cached, rows)]
    st["ts_offsets"] = _offsets(n)
    gap = torch.empty(sum(n), device=DEV, dtype=torch.float64).exponential_(1 / 600.0, generator=g).round().clamp(min=1).long()
    ts = []
    for u in range(c["B"]):
        a, e = int(sum(n[:u])), int(sum(n[:u + 1]))
        t = 1_700_000_000 + torch.cumsum(gap[a:e], 0)
        w = min(c["cand"], rows[u])
        if 0 < w < len(t):
            t[len(t) - w:] = t[len(t) - w - 1]
        elif w:
            t[:] = t[0]
        ts.append(t)
    st["ts"] = torch.cat(ts) if sum(n) else torch.zeros(0, dtype=torch.int64, device=DEV)
    st["rab_pos"] = 0.02 * _rand(g, 2 * c["n_max"] - 1)
    st["rab_ts"] = 0.02 * _rand(g, N_BUCKETS)
    st["gamma"] = 1 + 0.1 * _rand(g, hd)
    st["beta"] = 0.1 * _rand(g, hd)
    at = torch.arange(total, device=DEV)
    st["row_user"] = torch.searchsorted(st["offsets"].long(), at, right=True) - 1
    st["row_at"] = at - st["offsets"].long()[st["row_user"]]
    return st


# ---------------------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------------------
def run(st):
    c = st["c"]
    if c["op"] == "linear":
        return _own_linear(st) if own else _plain_linear(st)
    if c["op"] == "append":
        st["live"].copy_(st["ints"])  # the same append again
        k, v = _own_append(st) if own else _plain_append(st)
        return {"k": k, "v": v, "table": st["table"], "lens": st["lens"], "count": st["count"]}
    return _own_attn(st) if own else _plain_attn(st)


def _workspace(st, size, *args, **kw):
    """The scratch buffer that a program keeps beside its inputs, sized by the library at the first pass."""
    if "ws" not in st:
        st["ws"] = torch.empty(size(*args, **kw), dtype=torch.uint8, device=DEV)
    return st["ws"]


def _own_linear(st):
    import generative_recommender_attention_jagged_b200 as m
    c = st["c"]
    ws = _workspace(st, m.hstu_linear_i8_workspace_size, c["T"], c["K"], c["N"])
    return m.hstu_linear_i8(st["x"], st["w_q"], st["w_scale"], st["bias"], silu=c["silu"], out_dtype=DT[c["out"]],
                            workspace=ws)


def _own_append(st):
    import generative_recommender_attention_jagged_b200 as m
    ws = _workspace(st, m.hstu_kv_q4_workspace_size, st["c"]["B"])
    pools = (st["k_pool"], st["v_pool"], st["k_meta"], st["v_meta"])
    m.hstu_kv_append_q4(st["k"], st["v"], st["offsets"], *pools, st["table"], st["lens"], st["free"], st["count"],
                        workspace=ws)
    return m.hstu_kv_read_q4(*pools, st["table"], st["lens"], st["starts"], st["offsets"], total_tokens=st["total"],
                             dtype=st["k"].dtype, workspace=ws)


def _own_attn(st):
    import generative_recommender_attention_jagged_b200 as m
    c = st["c"]
    ws = _workspace(st, m.hstu_attn_paged_q4_workspace_size, batch=c["B"], num_heads=c["H"], head_dim=c["d"],
                    n_max=c["n_max"], total_tokens=st["total"], dtype=st["q"].dtype, max_cached_len=st["max_cached"])
    return m.hstu_attn_fwd_paged_q4(
        st["q"], st["k"], st["v"], st["u"], st["offsets"], st["ts"], st["ts_offsets"], st["rab_pos"], st["rab_ts"],
        st["k_pool"], st["v_pool"], st["k_meta"], st["v_meta"], st["table"], st["lens"], n_max=c["n_max"],
        num_candidates=st["cand"], ln_gamma=st["gamma"], ln_beta=st["beta"], max_cached_len=st["max_cached"],
        workspace=ws)


def _plain_linear(st):
    c = st["c"]
    x = st["x"].float()
    amax = x.abs().amax(1)
    scale = amax / torch.full_like(amax, 127.0)
    scale = torch.where(scale >= TINY, scale, torch.zeros_like(scale))
    use = torch.where(scale > 0, scale, torch.ones_like(scale))
    code = (x.double() / use.double()[:, None]).round().clamp(-127, 127)
    code = torch.where(scale[:, None] > 0, code, torch.zeros_like(code))
    # sums of up to 1024 products of two codes are exact in 32 bits, longer ones in 64
    num = torch.float32 if c["K"] <= 1024 else torch.float64
    acc = (code.to(num) @ st["w_q"].to(num).t()).float()
    y = acc * (scale[:, None] * st["w_scale"])
    if st["bias"] is not None:
        y = y + st["bias"]
    if c["silu"]:
        y = _silu(y)
    return y.to(DT[c["out"]])


def _plain_append(st):
    c, page = st["c"], st["c"]["page"]
    table, lens, count, off = st["table"], st["lens"], st["count"], st["offsets"].long()
    new = off[1:] - off[:-1]
    old = lens.long()
    have = (old + page - 1) // page
    need = (old + new + page - 1) // page - have
    before = torch.cumsum(need, 0) - need
    # user u's j-th new page comes from the top of the stack, users in order
    j = torch.arange(table.shape[1], device=DEV)[None, :] - have[:, None]
    take = (j >= 0) & (j < need[:, None])
    top = count.long() - 1 - before[:, None] - j
    table.copy_(torch.where(take, st["free"][top.clamp(0, st["pages"] - 1)], table))
    lens.add_(new.to(torch.int32))
    count.sub_(need.sum().to(torch.int32))
    at = torch.arange(st["total"], device=DEV)
    user = torch.searchsorted(off, at, right=True) - 1
    pos = old[user] + at - off[user]
    pid = table[user, pos // page].long()
    got = []
    for x in ("k", "v"):  # the two halves of the cache
        code, s, z = _quant4(st[x].float())
        st[x + "_pool"][pid, :, pos % page] = _pack4(code)
        st[x + "_meta"][pid, :, pos % page] = torch.stack([s, z], -1)
        got.append(_dequant4(st[x + "_pool"][pid, :, pos % page], st[x + "_meta"][pid, :, pos % page]).to(st[x].dtype))
    return got


def _plain_attn(st):
    c = st["c"]
    b, h, d, page, n_max = c["B"], c["H"], c["d"], c["page"], c["n_max"]
    rows, keys = st["max_rows"], st["max_cached"] + st["max_rows"]
    off, lens = st["offsets"].long(), st["lens"].long()
    new = off[1:] - off[:-1]
    n = lens + new
    cand = st["cand"].long() if st["cand"] is not None else torch.zeros_like(n)
    hist = n - cand
    pos = torch.arange(keys, device=DEV)
    slot = pos // page
    pid = st["table"][:, slot.clamp(max=st["table"].shape[1] - 1)].clamp(min=0).long()  # [b, keys]
    cached = pos[None] < lens[:, None]
    fresh = (off[:-1, None] + pos[None] - lens[:, None]).clamp(0, st["total"] - 1)
    used = pos[None] < n[:, None]

    def rows_of(x):  # [b, h, keys, d]: the cached rows, then the new ones, nothing behind the last
        old = _dequant4(st[x + "_pool"][pid, :, (pos % page)[None].expand_as(pid)],
                        st[x + "_meta"][pid, :, (pos % page)[None].expand_as(pid)])
        both = torch.where(cached[:, :, None, None], old, st[x][fresh].float())
        return torch.where(used[:, :, None, None], both, torch.zeros_like(both)).transpose(1, 2)

    r = torch.arange(rows, device=DEV)
    i = lens[:, None] + r[None]  # [b, rows]: positions of the new rows
    q = st["q"][(off[:-1, None] + r[None]).clamp(0, st["total"] - 1)].float().transpose(1, 2)
    s = (q @ rows_of("k").transpose(2, 3)) * (1.0 / math.sqrt(d))
    pi, pj = torch.minimum(i, hist[:, None]), torch.minimum(pos[None], hist[:, None])
    at = (pi[:, :, None] - pj[:, None, :] + n_max - 1).clamp(0, 2 * n_max - 2)
    tsb = st["ts_offsets"].long()[:-1, None]
    last = st["ts"].numel() - 1
    dt = (st["ts"][(tsb + i).clamp(max=last)][:, :, None] - st["ts"][(tsb + pos[None]).clamp(max=last)][:, None, :]).abs()
    bucket = torch.floor(torch.log(dt.double() + 1) / 0.301).long().clamp(0, N_BUCKETS - 1)
    s = s + (st["rab_pos"][at] + st["rab_ts"][bucket])[:, None]
    ok = torch.where(i[:, :, None] < hist[:, None, None], pos <= i[:, :, None],
                     (pos < hist[:, None, None]) | (pos == i[:, :, None])) & used[:, None, :]
    a = torch.where(ok[:, None], _silu(s), torch.zeros_like(s)) / n_max
    o = (a @ rows_of("v")).transpose(1, 2).flatten(2)[st["row_user"], st["row_at"]]
    mean = o.mean(1, keepdim=True)
    var = (o - mean).square().mean(1, keepdim=True)
    y = ((o - mean) / torch.sqrt(var + EPS) * st["gamma"] + st["beta"]) * st["u"].float()
    return y.to(st["q"].dtype)


# ---------------------------------------------------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------------------------------------------------
def _exact_rows(byte, meta):
    """Bytes [m, h, d / 2] and (scale, zero) [m, h, 2] -> [m, h, d] in 64 bits, a nibble at a time."""
    w = byte.long().unflatten(-1, (-1, 4))
    word = w[..., 0] + 256 * w[..., 1] + 65536 * w[..., 2] + 16777216 * w[..., 3]
    out = torch.zeros(*word.shape, 8, dtype=torch.float64, device=byte.device)
    for e in range(8):
        nib = (e // 2) + 4 * (e % 2)
        out[..., e] = (word // 16 ** nib % 16).double()
    return (out.flatten(-2) - meta[..., 1:].double()) * meta[..., :1].double()


def exact(c, seed):
    global own
    was, own = own, False
    try:
        st = prepare(c, seed)
    finally:
        own = was
    if c["op"] == "linear":
        outs = []
        wq = st["w_q"].double() * st["w_scale"].double()[:, None]
        for t0 in range(0, c["T"], 4096):
            x = st["x"][t0:t0 + 4096].double()
            scale = (x.abs().max(1).values.float() / torch.tensor(127.0, device=DEV).expand(len(x))).double()
            x = torch.round(x / scale.clamp(min=1e-300)[:, None]) * scale[:, None]
            y = x @ wq.T
            if st["bias"] is not None:
                y = y + st["bias"].double()
            outs.append(y * torch.sigmoid(y) if c["silu"] else y)
        return torch.cat(outs)
    if c["op"] == "append":
        new, cached = _lengths(c)
        out = {}
        for x in ("k", "v"):
            v = st[x].double()
            lo = torch.minimum(v.min(-1, keepdim=True).values, torch.zeros((), device=DEV, dtype=torch.float64))
            hi = torch.maximum(v.max(-1, keepdim=True).values, torch.zeros((), device=DEV, dtype=torch.float64))
            s = ((hi - lo).float() / torch.tensor(15.0, device=DEV).expand_as(lo)).bfloat16().double()
            z = torch.round(-lo / s)
            out[x] = s * (torch.clamp(torch.round(v / s) + z, 0, 15) - z.clamp(0, 15))
        page = c["page"]
        table, lens, count = st["table"].clone(), [], int(st["count"][0])
        for u in range(c["B"]):
            for p in range(-(-cached[u] // page), -(-(cached[u] + new[u]) // page)):
                count -= 1
                table[u, p] = st["free"][count]
            lens.append(cached[u] + new[u])
        return {**out, "table": table, "lens": torch.tensor(lens, dtype=torch.int32), "count": torch.tensor([count], dtype=torch.int32)}
    h, d, page, n_max = c["H"], c["d"], c["page"], c["n_max"]
    outs = []
    for u in range(c["B"]):
        r, l = st["rows"][u], st["cached"][u]
        if r == 0:
            continue
        a0, t0 = int(sum(st["rows"][:u])), int(st["ts_offsets"][u])
        n, cn = l + r, min(c["cand"], r)
        hist = n - cn
        key, val = (st[x][a0:a0 + r].double() for x in ("k", "v"))
        if l:
            j = torch.arange(l, device=DEV)
            p = st["table"][u, j // page].long()
            key = torch.cat([_exact_rows(st["k_pool"][p, :, j % page], st["k_meta"][p, :, j % page]), key])
            val = torch.cat([_exact_rows(st["v_pool"][p, :, j % page], st["v_meta"][p, :, j % page]), val])
        s = torch.einsum("ihd,jhd->hij", st["q"][a0:a0 + r].double(), key) / math.sqrt(d)
        j = torch.arange(n, device=DEV)
        i = j[l:, None]
        s += st["rab_pos"].double()[i.clamp(max=hist) - j.clamp(max=hist) + n_max - 1]
        t = st["ts"][t0:t0 + n]
        gap = (t[l:, None] - t[None]).abs().double()
        s += st["rab_ts"].double()[(torch.log1p(gap) / 0.301).floor().clamp(0, N_BUCKETS - 1).long()]
        seen = ((i < hist) & (j <= i)) | ((i >= hist) & ((j < hist) | (j == i)))
        o = torch.einsum("hij,jhd->ihd", torch.sigmoid(s) * s * seen, val).reshape(r, h * d) / n_max
        o = (o - o.mean(1, keepdim=True)) * torch.rsqrt(o.var(1, unbiased=False, keepdim=True) + EPS)
        outs.append((o * st["gamma"].double() + st["beta"].double()) * st["u"][a0:a0 + r].double())
    return torch.cat(outs)
