"""Paged key/value cache operators: the cases they are measured on, in plain
form and through the framework.

``kv_cache_append`` rotates new queries and keys by their positions and writes
keys and values into the blocks of a paged cache (bf16, or e4m3 with a scale
for each block of tokens and head).  ``kv_cache_attention`` is the causal,
optionally windowed grouped-query attention of the newest tokens of each
sequence over that cache.

A case names an operator ("op"), the batch, the padded number of new tokens S
(ragged: each sequence has its own number of them), the context lengths
("ctx" is the longest; "spread" the shortest's share of it), heads, head
size, tokens per block, the cache's type and the window (0: none).
"""
import random

import torch

own = False

E4M3_MAX = 448.0
MIN_SCALE = 2.0 ** -64


def _case(name, op, B, S, ctx, spread, hq, hkv, d, block, cache, window=0, ragged=False,
          interleaved=False):
    c = {"op": op, "B": B, "S": S, "ctx": ctx, "spread": spread, "hq": hq, "hkv": hkv, "d": d,
         "block": block, "cache": cache, "window": window, "ragged": ragged,
         "interleaved": interleaved}
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one step of a batch that is answering: 64 sequences get a token each
        _case("append_step", "append", 64, 1, 500, 0.02, 32, 8, 128, 64, "e4m3"),
        # the prompt of the sliding-window workload goes into the cache at once
        _case("append_prompt", "append", 1, 32768, 32768, 1.0, 32, 8, 128, 64, "e4m3"),
        # padded pieces of prompts of several users, unquantised, pairs side by side
        _case("append_pieces", "append", 7, 777, 1501, 0.6, 16, 16, 64, 16, "bf16", ragged=True,
              interleaved=True),
        # one user: the latency of a single answer
        _case("decode_one", "attend", 1, 1, 4096, 1.0, 32, 8, 128, 64, "e4m3"),
        # a full batch with contexts of every length
        _case("decode_batch", "attend", 64, 1, 8192, 0.05, 32, 8, 128, 64, "e4m3"),
        # few users with very long documents
        _case("decode_long", "attend", 2, 1, 131071, 0.9, 32, 8, 128, 64, "e4m3"),
        # no shared heads, the smaller head size, short blocks, unquantised
        _case("decode_heads", "attend", 24, 1, 4001, 0.1, 16, 16, 64, 16, "bf16"),
        # the sliding window of 4096 tokens at its full sequence length
        _case("decode_window", "attend", 16, 1, 32768, 0.5, 32, 8, 128, 64, "e4m3", window=4096),
        # one key head for all queries
        _case("decode_shared", "attend", 8, 1, 16384, 0.3, 32, 1, 64, 128, "e4m3"),
        # drafted tokens are checked, five at a time
        _case("draft_check", "attend", 16, 5, 8192, 0.3, 32, 8, 128, 32, "e4m3"),
        # a long prompt comes in pieces: the newest piece reads what is there
        _case("chunk_long", "attend", 1, 2048, 32768, 1.0, 32, 8, 128, 64, "e4m3"),
        # padded pieces of several prompts, unquantised, windowed
        _case("chunk_pieces", "attend", 4, 511, 6000, 0.2, 32, 8, 128, 128, "bf16", window=4096,
              ragged=True),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


HEADS = ((32, 8), (16, 16), (32, 1), (16, 4), (8, 8), (24, 2), (12, 4))


def draw(rng):
    op = rng.choice(("append", "attend", "attend"))
    hq, hkv = rng.choice(HEADS)
    d = rng.choice((64, 128))
    block = rng.choice((16, 32, 64, 128))
    cache = rng.choice(("e4m3", "e4m3", "bf16"))
    interleaved = rng.random() < 0.3
    spread = round(rng.uniform(0.02, 1.0), 3)
    if op == "append":
        B = _log_uniform(rng, 1, 64)
        S = 1 if rng.random() < 0.4 else _log_uniform(rng, 2, max(2, 32768 // B))
        ctx = S + _log_uniform(rng, 1, 512)
        return _case("", op, B, S, ctx, spread, hq, hkv, d, block, cache, 0, S > 1, interleaved)
    kind = rng.choice(("one", "few", "many"))
    window = _log_uniform(rng, 16, 8192) if rng.random() < 0.4 else 0
    if kind == "many":
        S = _log_uniform(rng, 17, 2048)
        B = _log_uniform(rng, 1, max(1, min(8, 2048 // S)))
        ctx = S + _log_uniform(rng, 64, 24576)
    else:
        S = 1 if kind == "one" else rng.randint(2, 16)
        B = _log_uniform(rng, 1, 64)
        most = 2 * 131072 * 8 * 128 // (B * hkv * d * (2 if cache == "bf16" else 1))
        ctx = S + _log_uniform(rng, 64, max(64, min(131072, most) - S))
    return _case("", op, B, S, ctx, spread, hq, hkv, d, block, cache, window, S > 1, False)


def _lengths(c):
    """(tokens in the cache with the new ones, new tokens) of each sequence."""
    rng = random.Random(1000003 * c["B"] + 1009 * c["S"] + c["ctx"])
    lens, new = [], []
    for b in range(c["B"]):
        n = c["S"] if not c["ragged"] or b == 0 else rng.randint(1, c["S"])
        low = max(n, int(c["ctx"] * c["spread"]))
        lens.append(c["ctx"] if b == 0 else rng.randint(low, max(low, c["ctx"])))
        new.append(n)
    return lens, new


def _scale_for(amax):
    """The smallest power of two s with amax <= 448 s."""
    e = torch.ceil(torch.log2(amax.double().clamp_min(1e-300) / E4M3_MAX))
    return torch.exp2(e).clamp_min(MIN_SCALE).float()


def _filled(shape, gen, cache, chunk=64):
    """A cache with something in every slot, and its scales: channels and heads
    differ in size, as keys and values do."""
    nb, h, bs, d = shape
    data = torch.empty(shape, dtype=torch.bfloat16 if cache == "bf16" else torch.float8_e4m3fn,
                       device="cuda")
    scale = torch.empty((nb, h), device="cuda")
    size = torch.exp(0.4 * torch.randn((h, 1, d), generator=gen, device="cuda"))
    for i in range(0, nb, chunk):
        n = min(chunk, nb - i)
        x = torch.randn((n, h, bs, d), generator=gen, device="cuda") * size
        if cache == "bf16":
            data[i:i + n] = x
        else:
            s = _scale_for(x.abs().amax(dim=(2, 3)))
            scale[i:i + n] = s
            data[i:i + n] = (x / s[:, :, None, None]).to(torch.float8_e4m3fn)
    return data, (scale if cache == "e4m3" else None)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    lens, new = _lengths(c)
    bs = c["block"]
    per = [-(-n // bs) for n in lens]
    nb, width = sum(per) + 3, max(per)
    order = torch.randperm(nb, generator=gen, device="cuda").to(torch.int32)
    table = torch.zeros((c["B"], width), dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = order[at:at + n]
        at += n
    shape = (nb, c["hkv"], bs, c["d"])
    chunk = max(1, (1 << 26) // (c["hkv"] * bs * c["d"]))
    kc, ks = _filled(shape, gen, c["cache"], chunk)
    vc, vs = _filled(shape, gen, c["cache"], chunk)
    s = {"case": c, "k_cache": kc, "v_cache": vc, "k_scale": ks, "v_scale": vs,
         "block_table": table,
         "seq_lens": torch.tensor(lens, dtype=torch.int32, device="cuda"),
         "new_lens": torch.tensor(new, dtype=torch.int32, device="cuda") if c["ragged"] else None}

    def tokens(heads):
        x = torch.randn((c["B"], c["S"], heads, c["d"]), generator=gen, device="cuda")
        return x.to(torch.bfloat16).transpose(1, 2)     # as a projection's output is seen

    s["q"] = tokens(c["hq"])
    if c["op"] == "append":
        s["k"], s["v"] = tokens(c["hkv"]), tokens(c["hkv"])
        pos = torch.arange(width * bs, device="cuda", dtype=torch.float64)
        freq = 10000.0 ** (-torch.arange(0, c["d"], 2, device="cuda", dtype=torch.float64) / c["d"])
        ang = pos[:, None] * freq[None, :]
        s["rope"] = torch.cat([ang.cos(), ang.sin()], dim=1).float()
        # rows of padding are not written: their place in the output is known
        s["q_out"] = torch.zeros((c["B"], c["hq"], c["S"], c["d"]), dtype=torch.bfloat16,
                                 device="cuda")
    else:
        s["out"] = torch.zeros((c["B"], c["hq"], c["S"], c["d"]), dtype=torch.bfloat16,
                               device="cuda")
    return s


def run(state):
    s = state
    c = s["case"]
    if own:
        import block_sparse_local_b200 as sta
        if c["op"] == "append":
            q = sta.kv_cache_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["block_table"],
                                    s["seq_lens"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                                    new_lens=s["new_lens"], q=s["q"], rope=s["rope"],
                                    interleaved=c["interleaved"], q_out=s["q_out"])
            return _appended(s, q)
        return sta.kv_cache_attention(s["q"], s["k_cache"], s["v_cache"], s["block_table"],
                                      s["seq_lens"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                                      new_lens=s["new_lens"], window=c["window"], out=s["out"])
    if c["op"] == "append":
        return _appended(s, _plain_append(s))
    return _plain_attend(s)


def _appended(s, q):
    """The rotated queries and the updated cache: e4m3 numbers stand for
    themselves times the scale of their block and head, which comes with them."""
    r = {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if s["k_scale"] is not None:
        r["k_scale"], r["v_scale"] = s["k_scale"], s["v_scale"]
    return r


def _positions(s):
    c = s["case"]
    step = torch.arange(c["S"], device="cuda")
    new = s["new_lens"].long() if s["new_lens"] is not None else \
        torch.full((c["B"],), c["S"], device="cuda")
    pos = (s["seq_lens"].long() - new)[:, None] + step[None, :]
    return pos, (step[None, :] < new[:, None]) & (pos >= 0)


def _plain_rotate(x, pos, rope, interleaved):
    half = x.shape[-1] // 2
    cs = rope[pos.clamp(0, rope.shape[0] - 1)][:, None]      # [B, 1, S, d]
    cos, sin = cs[..., :half], cs[..., half:]
    x = x.float()
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :half], x[..., half:])
    y = (a * cos - b * sin, b * cos + a * sin)
    return torch.stack(y, -1).flatten(-2) if interleaved else torch.cat(y, -1)


def _plain_append(s):
    c = s["case"]
    pos, valid = _positions(s)
    q = _plain_rotate(s["q"], pos, s["rope"], c["interleaved"]).to(torch.bfloat16)
    s["q_out"].copy_(torch.where(valid[:, None, :, None], q, s["q_out"]))
    bs = c["block"]
    entry = (pos // bs).clamp(0, s["block_table"].shape[1] - 1)     # padding's too: not used
    block = torch.gather(s["block_table"].long(), 1, entry)[valid]
    slot = (pos % bs)[valid]
    _plain_store(_plain_rotate(s["k"], pos, s["rope"], c["interleaved"]).transpose(1, 2)[valid],
                 s["k_cache"], s["k_scale"], block, slot)
    _plain_store(s["v"].float().transpose(1, 2)[valid], s["v_cache"], s["v_scale"], block, slot)
    return s["q_out"]


def _plain_store(x, cache, scale, block, slot):
    """Tokens x [n, heads, d] into (block, slot) of the cache."""
    if scale is None:
        cache[block, :, slot] = x.to(torch.bfloat16)
        return
    nb, h, bs, _ = cache.shape
    finite = torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x)).amax(-1)
    amax = torch.zeros((nb, h), device="cuda").index_reduce_(0, block, finite, "amax")
    first = torch.full((nb,), bs, device="cuda").index_reduce_(0, block, slot, "amin")
    touched, fresh = (first < bs)[:, None], (first == 0)[:, None]
    need = _scale_for(amax)
    grown = torch.where(fresh, need, torch.maximum(scale, need))
    ratio = torch.where(touched & ~fresh, scale / grown, 1.0)
    earlier = torch.arange(bs, device="cuda")[None, :] < first[:, None]
    move = touched & ~fresh & (ratio < 1.0)
    moved = (cache.float() * ratio[:, :, None, None]).to(torch.float8_e4m3fn)
    old = move[:, :, None, None] & earlier[:, None, :, None]
    raw = cache.view(torch.uint8)
    raw.copy_(torch.where(old, moved.view(torch.uint8), raw))
    scale.copy_(torch.where(touched, grown, scale))
    code = (x / scale[block][..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    raw[block, :, slot] = code.view(torch.uint8)


def _plain_attend(s):
    c = s["case"]
    B, hq, S, d = s["q"].shape
    hkv = c["hkv"]

    def gathered(cache, scale):
        table = s["block_table"].long()
        x = cache.view(torch.uint8 if scale is not None else cache.dtype)[table]
        x = x.view(cache.dtype).float()                       # [B, nb, hkv, block, d]
        if scale is not None:
            x = x * scale[table][..., None, None]
        return x.transpose(1, 2).reshape(B, hkv, -1, d)

    k = gathered(s["k_cache"], s["k_scale"])
    L = k.shape[2]
    pos, valid = _positions(s)
    key = torch.arange(L, device="cuda")
    there = key[None, :] < s["seq_lens"].long()[:, None]      # [B, L]
    see = (key[None, None, :] <= pos[:, :, None]) & valid[:, :, None] & there[:, None, :]
    if c["window"]:
        see &= key[None, None, :] > pos[:, :, None] - c["window"]
    q = s["q"].float().reshape(B, hkv, (hq // hkv) * S, d)
    p = torch.matmul(q, k.transpose(2, 3)).reshape(B, hq, S, L)
    del k
    p *= d ** -0.5
    p.masked_fill_(~see[:, None], float("-inf"))
    top = p.amax(-1, keepdim=True)
    p -= torch.where(torch.isinf(top), torch.zeros_like(top), top)
    p.exp_()
    total = p.sum(-1, keepdim=True)
    v = gathered(s["v_cache"], s["v_scale"])
    v.masked_fill_(~there[:, None, :, None], 0.0)
    o = torch.matmul(p.reshape(B, hkv, (hq // hkv) * S, L), v).reshape(B, hq, S, d)
    o = torch.where(total > 0, o / total, torch.zeros_like(o)).to(torch.bfloat16)
    s["out"].copy_(torch.where(valid[:, None, :, None], o, s["out"]))
    return s["out"]


def work(case):
    c = case
    lens, new = _lengths(c)
    row = 2 * c["d"]                                          # bytes of a bf16 row
    held = c["d"] * (2 if c["cache"] == "bf16" else 1)        # of a cached row
    scales = 0 if c["cache"] == "bf16" else 8
    tokens = sum(new)
    if c["op"] == "append":
        by = tokens * (2 * c["hq"] * row + 2 * c["hkv"] * (row + held) + 4 * c["d"])
        by += c["hkv"] * scales * sum(-(-n // c["block"]) for n in new)
        return {"bytes": by, "flops": 3 * tokens * (c["hq"] + c["hkv"]) * c["d"]}
    by = 2 * tokens * c["hq"] * row
    pairs = 0
    for n, s in zip(lens, new):
        seen = n if not c["window"] else min(n, c["window"] + s - 1)
        by += c["hkv"] * (2 * held * seen + scales * -(-seen // c["block"]) + 4)
        first = n - s
        if c["window"]:
            pairs += sum(min(first + i + 1, c["window"]) for i in range(s))
        else:
            pairs += s * first + s * (s + 1) // 2
    return {"bytes": by, "flops": 4 * pairs * c["hq"] * c["d"]}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    """The same from the definitions, one sequence after another, in 64 bits.
    e4m3 numbers are left unrounded: the quotient that the number stands for."""
    s = prepare(case, seed)
    return _exact_append(s) if case["op"] == "append" else _exact_attend(s)


def _turn(x, p, table, side_by_side):
    """x [heads, n, d] turned by the angles of positions p, as complex numbers."""
    half = x.shape[-1] // 2
    w = torch.complex(table[p, :half].double(), table[p, half:].double())
    if side_by_side:
        z = torch.view_as_complex(x.double().reshape(*x.shape[:-1], half, 2).contiguous()) * w
        return torch.view_as_real(z).flatten(-2)
    z = torch.complex(x[..., :half].double(), x[..., half:].double()) * w
    return torch.cat([z.real, z.imag], -1)


def _exact_append(s):
    c = s["case"]
    lens, new = _lengths(c)
    bs = c["block"]
    q = s["q_out"].double()
    r = {n: s[n].double() for n in ("k_cache", "v_cache")}
    held = {n: (s[n].double() if s[n] is not None else None) for n in ("k_scale", "v_scale")}
    for b in range(c["B"]):
        n = new[b]
        p = torch.arange(lens[b] - n, lens[b], device="cuda")
        q[b, :, :n] = _turn(s["q"][b, :, :n], p, s["rope"], c["interleaved"])
        k = _turn(s["k"][b, :, :n], p, s["rope"], c["interleaved"])
        v = s["v"][b, :, :n].double()
        # the blocks that get tokens, as one row of slots
        i0, i1 = (lens[b] - n) // bs, (lens[b] - 1) // bs + 1
        ids = s["block_table"][b, i0:i1].long()
        lead = (lens[b] - n) - i0 * bs
        for name, x in (("k", k), ("v", v)):
            data = r[name + "_cache"]
            view = data[ids].transpose(0, 1).reshape(c["hkv"], -1, c["d"])   # [h, slots, d]
            if c["cache"] == "bf16":
                view[:, lead:lead + n] = x
            else:
                scale = held[name + "_scale"]
                room = torch.zeros((c["hkv"], (i1 - i0) * bs), device="cuda", dtype=torch.float64)
                room[:, lead:lead + n] = x.abs().amax(-1)
                most = room.reshape(c["hkv"], i1 - i0, bs).amax(-1)          # [h, blocks]
                m, e = torch.frexp(most / E4M3_MAX)                          # m in [1/2, 1)
                want = torch.ldexp(torch.ones_like(most), torch.where(m == 0.5, e - 1, e))
                was = scale[ids].transpose(0, 1)
                now = want.clamp_min(MIN_SCALE)
                if lead:
                    now[:, 0] = torch.maximum(now[:, 0], was[:, 0])
                    view[:, :lead] *= (was[:, 0] / now[:, 0])[:, None, None]
                view[:, lead:lead + n] = x / now.repeat_interleave(bs, 1)[:, lead:lead + n, None]
                scale[ids] = now.transpose(0, 1)
            data[ids] = view.reshape(c["hkv"], i1 - i0, bs, c["d"]).transpose(0, 1)
    r["q"] = q
    if c["cache"] == "e4m3":
        r.update(held)
    return r


def _exact_attend(s):
    c = s["case"]
    lens, new = _lengths(c)
    bs, group = c["block"], c["hq"] // c["hkv"]
    out = s["out"].double()
    for b in range(c["B"]):
        n, L = new[b], lens[b]
        lo = max(0, L - n - c["window"] + 1) // bs * bs if c["window"] else 0
        ids = s["block_table"][b, lo // bs:-(-L // bs)].long()
        p = torch.arange(L - n, L, device="cuda")
        j = torch.arange(lo, L, device="cuda")
        hide = j[None, :] > p[:, None]
        if c["window"]:
            hide |= j[None, :] <= p[:, None] - c["window"]
        for h in range(c["hkv"]):
            kv = []
            for data, scale in ((s["k_cache"], s["k_scale"]), (s["v_cache"], s["v_scale"])):
                x = data[:, h].view(torch.uint8)[ids].view(data.dtype).double()
                if scale is not None:
                    x = x * scale[ids, h].double()[:, None, None]
                kv.append(x.reshape(-1, c["d"])[:L - lo])
            for g in range(h * group, (h + 1) * group):
                w = (s["q"][b, g, :n].double() @ kv[0].T) / c["d"] ** 0.5
                out[b, g, :n] = torch.softmax(w.masked_fill(hide, float("-inf")), -1) @ kv[1]
    return out
