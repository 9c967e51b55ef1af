"""Paged cache, storing tokens: sta_kv_append against the float64 oracle.

Roundings.  A rotated value is two products and a sum in fp32, each off by at
most 2^-24 relative: |error| <= 2 * 2^-24 (|a| + |b|) =: r.  It is then rounded
once: to bf16 (2^-8 of the value) or to e4m3 (2^-4 of the value in the normal
range, 2^-10 of the scale below it).  Unrotated values reach that rounding
unchanged, so values of an e4m3 cache equal the oracle's exactly; so do scales,
as long as no block's largest rotated value lies within r of 448 times a power
of two (none does with these seeds).
"""
import numpy as np
import pytest
import torch

import block_sparse_local_b200 as sta
from oracle import kv_oracle
from tests import kv_cases

pytestmark = pytest.mark.gpu
R = 2.0 ** -23


def _raw(x):
    return x.view(torch.uint8 if x.dtype == torch.float8_e4m3fn else torch.int16)


def check_append(rng, lens, new, S, hq, hkv, d, block, quant, inter=False, rope=True, std=None,
                 spoil=None, strided=True, in_place=False):
    B = len(lens)
    t, ref, table = kv_cases.rand_cache(rng, lens, hkv, d, block, quant, junk=False)
    # rows as a projection leaves them: [B, S, heads, d]
    k, v, q = (kv_cases.bf16(rng, (B, S, h, d)) for h in (hkv, hkv, hq))
    if std is not None:
        k, v = (k.float() * std).to(torch.bfloat16), (v.float() * std).to(torch.bfloat16)
    if spoil is not None:
        spoil(k, v)
    k, v, q = (x.transpose(1, 2) for x in (k, v, q))
    if not strided:
        k, v, q = (x.contiguous() for x in (k, v, q))
    width = table.shape[1]
    rows = width * block + 3
    tab = sta.rope_table(rows, d) if rope else None
    before = kv_cases.cuda(t)
    g = {n: (x.clone() if x is not None else None) for n, x in before.items()}
    qg = q.cuda() if rope else None
    fill = torch.full((B, hq, S, d), 7.0, dtype=torch.bfloat16, device="cuda")
    q_out = None if not rope else (qg.clone() if in_place else fill)
    got = sta.kv_cache_append(
        k.cuda(), v.cuda(), g["k_cache"], g["v_cache"], kv_cases.i32(table), kv_cases.i32(lens),
        k_scale=g["k_scale"], v_scale=g["v_scale"],
        new_lens=None if new is None else kv_cases.i32(new),
        q=q_out if in_place and rope else qg, rope=tab, interleaved=inter, q_out=q_out)
    torch.cuda.synchronize()
    sta._check(sta.lib().sta_device_status(None), "status")

    kd, vd, qd = (x.double().numpy() for x in (k, v, q))
    tabd = tab.cpu().double().numpy() if rope else None
    kv_oracle.append(ref, kd, vd, table, lens, new, tabd, inter, quant, round_k=False)
    place = kv_oracle.positions(lens, new, S)

    # queries
    if rope:
        out = got.float().cpu().numpy()
        left = np.ones((B, S), dtype=bool)
        for b, s, p in place:
            left[b, s] = False
            want = kv_oracle.rotate(qd[b, :, s], p, tabd, inter)
            size = np.abs(qd[b, :, s]).max(-1, keepdims=True)
            assert (np.abs(out[b, :, s] - want) <= 2.0 ** -8 * np.abs(want) + 2 * R * size).all()
        kept = (q_out if not in_place else qg).float().cpu().numpy()
        for b, s in zip(*np.nonzero(left)):
            assert np.array_equal(out[b, :, s], kept[b, :, s], equal_nan=True)
    else:
        assert got is None

    # slots that the call does not store to: bits as they were, or (a grown
    # scale) the oracle's number
    nb = ref["k"].shape[0]
    stored = np.zeros((nb, block), dtype=bool)
    touched = np.zeros(nb, dtype=bool)
    for b, s, p in place:
        stored[table[b, p // block], p % block] = True
        touched[table[b, p // block]] = True
    for n in ("k", "v"):
        a, w = _raw(g[n + "_cache"]).cpu(), _raw(before[n + "_cache"]).cpu()
        other = torch.from_numpy(~touched)
        assert torch.equal(a[other], w[other])
        if quant:
            sc = g[n + "_scale"].double().cpu().numpy()
            assert np.array_equal(sc, ref[n + "s"])
        num = g[n + "_cache"].double().cpu().numpy()
        old = ~stored[:, None, :, None] & np.ones(num.shape, dtype=bool)
        # behind the last new token of a block that the call rescaled the numbers
        # are unspecified (nothing is there): only earlier slots are compared
        for b, s, p in place:
            blk, last = table[b, p // block], p % block
            old[blk, :, last:] = False
        assert np.array_equal(num[old], ref[n][old], equal_nan=True)
        new_ = np.broadcast_to(stored[:, None, :, None], num.shape)
        x, y = num[new_], ref[n][new_]
        if n == "v" or not rope:
            y = kv_oracle.e4m3_round(y) if quant else y
            assert np.array_equal(x, y, equal_nan=True)
        else:
            fin = np.isfinite(y) & (np.abs(y) <= 448.0 if quant else True)
            sz = 8.0 * (1.0 if std is None else std)
            s_ = ref["ks"][:, :, None, None] * np.ones(num.shape)
            r = 2 * R * sz / s_[new_]
            tol = r + (np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10) if quant
                       else 2.0 ** -8 * np.abs(y))
            assert (np.abs(x - y) <= tol)[fin].all()
            assert np.array_equal(np.isnan(x), np.isnan(y))
    return g, ref, table


CASES = [
    # lens, new, S, hq, hkv, d, block, interleaved
    ([1], None, 1, 4, 1, 64, 16, False),
    ([17, 16, 33], None, 1, 4, 2, 128, 16, True),
    ([64, 65, 128, 200], None, 1, 8, 8, 64, 64, False),
    ([300], None, 300, 4, 2, 128, 128, False),
    ([300], None, 300, 4, 2, 128, 128, True),
    ([70, 5, 40], [40, 5, 0], 40, 3, 3, 64, 32, True),
    ([129, 1, 0, 77], [129, 1, 0, 2], 129, 8, 4, 128, 64, False),
    ([0, 12, 3], [0, 3, 3], 3, 6, 2, 64, 16, False),
    # an unused place of the batch without new_lens: nothing stored, nothing rotated
    ([0, 9], None, 1, 4, 2, 128, 32, False),
    ([513], [511], 512, 32, 8, 128, 64, False),
]


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_append(case, quant):
    lens, new, S, hq, hkv, d, block, inter = case
    check_append(np.random.default_rng(100), lens, new, S, hq, hkv, d, block, quant, inter)


@pytest.mark.parametrize("quant", [False, True])
def test_without_rotation_and_queries(quant):
    check_append(np.random.default_rng(101), [50, 20], [33, 4], 33, 4, 2, 64, 16, quant,
                 rope=False)


@pytest.mark.parametrize("std", [1e-3, 40.0, 1e4])
def test_scale_grows_inside_a_block(std):
    # block numbers around 1 are already there; new ones are smaller or larger
    check_append(np.random.default_rng(102), [40, 9], [3, 2], 3, 4, 2, 128, 64, True, std=std)


def test_in_place_queries_and_contiguous_rows():
    check_append(np.random.default_rng(103), [40, 9], [3, 2], 3, 4, 2, 128, 64, True,
                 in_place=True, strided=False)


@pytest.mark.parametrize("quant", [False, True])
def test_infinities_and_nan_stay_in_their_place(quant):
    def spoil(k, v):
        v[0, 1, 0, 3] = float("inf")
        v[0, 1, 0, 4] = float("-inf")
        v[0, 2, 1, 5] = float("nan")
    check_append(np.random.default_rng(104), [40], [5], 5, 2, 2, 64, 16, quant, spoil=spoil)


def test_zeros_get_the_smallest_scale():
    g, ref, table = check_append(np.random.default_rng(105), [16], None, 16, 2, 2, 64, 16, True,
                                 std=0.0)
    assert (g["v_scale"][int(table[0, 0])] == 2.0 ** -64).all()


def test_values_of_every_size():
    # the scale's exponent over bf16's range, with 448 2^e at its border
    d, block = 64, 16
    for e in (-133, -100, -64, -60, -9, 0, 7, 100, 119):
        for m in (1.0, 1.75, 1.7578125):
            x = torch.zeros((1, 1, 1, d), dtype=torch.bfloat16)
            x[..., 0] = m * 2.0 ** e
            kc, vc, ks, vs = sta.kv_cache_empty(1, 1, block, d, dtype=torch.float8_e4m3fn)
            one = torch.ones(1, dtype=torch.int32, device="cuda")
            sta.kv_cache_append(x.cuda(), x.cuda(), kc, vc, torch.zeros_like(one)[None], one,
                                k_scale=ks, v_scale=vs)
            amax = float(x[..., 0].double())
            assert float(vs[0, 0]) == float(ks[0, 0]) == kv_oracle.e4m3_scale(amax)
            assert float(vc[0, 0, 0, 0].double()) == \
                kv_oracle.e4m3_round(amax / kv_oracle.e4m3_scale(amax))


def test_a_sequence_grows_token_by_token():
    # the cache after 40 single tokens equals the oracle's after the same calls
    rng = np.random.default_rng(106)
    d, block, H, n = 64, 16, 2, 40
    kc, vc, ks, vs = sta.kv_cache_empty(3, H, block, d, dtype=torch.float8_e4m3fn)
    ref = {x: np.zeros((3, H, block, d)) for x in ("k", "v")}
    ref.update({x: np.zeros((3, H)) for x in ("ks", "vs")})
    table = np.array([[2, 0, 1]])
    size = 2.0 ** rng.integers(-3, 4, n)
    for i in range(n):
        k, v = (kv_cases.bf16(rng, (1, H, 1, d), size[i]) for _ in range(2))
        sta.kv_cache_append(k.cuda(), v.cuda(), kc, vc, kv_cases.i32(table), kv_cases.i32([i + 1]),
                            k_scale=ks, v_scale=vs)
        kv_oracle.append(ref, k.double().numpy(), v.double().numpy(), table, [i + 1], None, None,
                         False, True)
    for got, want in ((kc, "k"), (vc, "v"), (ks, "ks"), (vs, "vs")):
        assert np.array_equal(got.double().cpu().numpy(), ref[want])


def test_strided_cache_heads_and_blocks():
    # K and V as one allocation, [block, K or V, head, ...]
    rng = np.random.default_rng(107)
    d, block, H = 128, 32, 3
    both = torch.zeros((4, 2, H, block, d), dtype=torch.bfloat16, device="cuda")
    k, v = (kv_cases.bf16(rng, (1, H, 50, d)) for _ in range(2))
    table = kv_cases.i32([[3, 1]])
    sta.kv_cache_append(k.cuda(), v.cuda(), both[:, 0], both[:, 1], table, kv_cases.i32([50]))
    for i, x in enumerate((k, v)):
        rows = both[:, i][[3, 1]].transpose(0, 1).reshape(H, 64, d)
        assert torch.equal(rows[:, :50].cpu(), x[0]) and not rows[:, 50:].any()
    assert not both[[0, 2]].any()


def test_bad_entries_are_reported_and_skipped():
    d, block = 64, 16
    k = torch.ones((3, 1, 1, d), dtype=torch.bfloat16, device="cuda")
    kc, vc, _, _ = sta.kv_cache_empty(2, 1, block, d)
    # a block outside the cache, a length behind the table, one good sequence
    for table, lens in (([[5], [1], [0]], [3, 17, 3]), ([[-1], [1], [0]], [3, 2 ** 31 - 1, 3]),
                        ([[2], [1], [0]], [16, 1000, 3])):
        kc.zero_(), vc.zero_()
        sta.kv_cache_append(k, k, kc, vc, kv_cases.i32(table), kv_cases.i32(lens))
        assert sta.lib().sta_device_status(None) == 6
        assert sta.lib().sta_device_status(None) == 0
        assert kc[0, 0, 2].eq(1).all() and kc.count_nonzero() == d and vc.count_nonzero() == d
    # negative lengths count as empty, too many new tokens as S
    kc.zero_()
    sta.kv_cache_append(k, k, kc, vc, kv_cases.i32([[5], [1], [0]]), kv_cases.i32([-4, 0, 2]),
                        new_lens=kv_cases.i32([1, -3, 9]))
    assert sta.lib().sta_device_status(None) == 0
    assert kc[0, 0, 1].eq(1).all() and kc.count_nonzero() == d


def test_other_stream_and_replayed_graph():
    # lengths are read on the device: one captured call stores the next token
    rng = np.random.default_rng(108)
    d, block, H = 64, 16, 2
    kc, vc, ks, vs = sta.kv_cache_empty(3, H, block, d, dtype=torch.float8_e4m3fn)
    want = [x.clone() for x in (kc, vc, ks, vs)]
    table = kv_cases.i32([[1, 2, 0]])
    toks = [tuple(kv_cases.bf16(rng, (1, H, 1, d)).cuda() for _ in range(2)) for _ in range(20)]
    k, v = (torch.zeros((1, H, 1, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    n = torch.zeros(1, dtype=torch.int32, device="cuda")
    tab = sta.rope_table(48, d)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        n.add_(1)
        sta.kv_cache_append(k, v, kc, vc, table, n, k_scale=ks, v_scale=vs, rope=tab)
    for x in (kc, vc, ks, vs, n):
        x.zero_()
    for i, (a, b) in enumerate(toks):
        k.copy_(a), v.copy_(b)
        g.replay()
        sta.kv_cache_append(a, b, *want[:2], table, kv_cases.i32([i + 1]), k_scale=want[2],
                            v_scale=want[3], rope=tab)
    torch.cuda.synchronize()
    for x, y in zip((kc, vc, ks, vs), want):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
