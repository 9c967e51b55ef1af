"""Paged cache, attention: sta_kv_attention against the float64 oracle.

Roundings.  out = sum_j w_j v_j / sum_j w_j over n keys.
- A score is a sum of d exact products, added in fp32 with truncation at worst:
  d 2^-23 of T = max_j |q| |k_j| / sqrt(d); as an exponent that is a relative
  error of w_j.  Its scaling and 2^x: below 2^-20 (T + 16) together, the argument
  (up to about T + 7 bits) being rounded at 2^-24 and ex2.approx good to 2^-22.
- Up to 64 query rows per key head and an e4m3 cache: a query's element is the sum
  of two e4m3 numbers, the largest of the row below 2^8, so off by half of e4m3's
  2^-9 at most, 2^-17 of the largest: 2^-17 max |q_i| |k|_1 / sqrt(d), which is
  below 2^-17 sqrt(d) T.
- w_j is rounded: to bf16 (2^-8) with a bf16 cache and more than 32 query rows; with
  fewer, to the sum of two bf16 numbers, the first at most a step (2^-7) below it
  and the second rounded (2^-15); to f16 (2^-11) with an e4m3 cache and many rows;
  with few, f16 and then three e5m2 numbers, of which the
  first two are cut off at 3 bits (leaving less than 2^-5 of the leading power of
  two, so a leading power below 2^-6 of it) and the last is rounded (half of 2^-2
  of its own): 2^-9 and 2^-11.  Weights below half of the last number (f16: 2^-25,
  e5m2: 2^-17) are lost, where the largest is above 2^7 (many rows), 2^10 (few).
- Numerator and denominator add n terms of one sign pattern each: n 2^-23.
So each weight is off by eps = d 2^-23 T + 2^-20 (T + 16) + P + n 2^-22 relative,
which moves out by at most 2 eps sum_j w_j |v_j| / sum_j w_j; the lost weights
move it by n 2^-32 (2^-27) max |v| at most; the result is rounded to bf16 (2^-8).
lse moves by eps without P.
"""
import numpy as np
import pytest
import torch

import block_sparse_local_b200 as sta
from oracle import kv_oracle
from tests import kv_cases

pytestmark = pytest.mark.gpu


def bounds(q, ref, spread, want, lens, quant):
    d = q.shape[-1]
    qn = np.linalg.norm(q, axis=-1).max()
    kn = np.linalg.norm(np.nan_to_num(ref["k"]) * ref["ks"][:, :, None, None], axis=-1).max()
    T = qn * kn / np.sqrt(d)
    n = max(lens)
    few = q.shape[1] // ref["k"].shape[1] * q.shape[2] <= 64
    eps = d * 2.0 ** -23 * T + 2.0 ** -20 * (T + 16) + n * 2.0 ** -22
    P = 2.0 ** -15 if q.shape[1] // ref["k"].shape[1] * q.shape[2] <= 32 else 2.0 ** -8
    vmax = np.abs(np.nan_to_num(ref["v"]) * ref["vs"][:, :, None, None]).max()
    lost = 0.0
    if quant:
        eps += 2.0 ** -17 * np.sqrt(d) * T if few else 0.0
        P = 2.0 ** -11 + (2.0 ** -9 if few else 0.0)
        lost = n * (2.0 ** -27 if few else 2.0 ** -32) * vmax
    return 2 * (eps + P) * spread + lost + 2.0 ** -8 * np.abs(want), eps


def check(rng, lens, new, S, hq, hkv, d, block, quant, window=0, q_std=1.0, layout="bshd",
          edit=None):
    B = len(lens)
    t, ref, table = kv_cases.rand_cache(rng, lens, hkv, d, block, quant)
    if edit is not None:
        edit(t, ref, table)
    q = kv_cases.bf16(rng, (B, S, hq, d), q_std).transpose(1, 2)
    if layout == "bhsd":
        q = q.contiguous()
    g = kv_cases.cuda(t)
    if layout == "sliced":                       # q as a part of a projection's row
        whole = torch.zeros((B, S, hq + 2 * hkv, d), dtype=torch.bfloat16, device="cuda")
        whole[:, :, :hq] = q.transpose(1, 2).cuda()
        qg = whole[:, :, :hq].transpose(1, 2)
        out = torch.full((B, S, hq + 1, d), 3.0, dtype=torch.bfloat16, device="cuda")[:, :, 1:]
        out = out.transpose(1, 2)
    else:
        qg = q.cuda() if layout == "bhsd" else q.transpose(1, 2).contiguous().cuda().transpose(1, 2)
        out = torch.full((B, hq, S, d), 3.0, dtype=torch.bfloat16, device="cuda")
    got, lse = sta.kv_cache_attention(
        qg, g["k_cache"], g["v_cache"], kv_cases.i32(table), kv_cases.i32(lens),
        k_scale=g["k_scale"], v_scale=g["v_scale"],
        new_lens=None if new is None else kv_cases.i32(new), window=window, out=out,
        return_lse=True)
    torch.cuda.synchronize()
    sta._check(sta.lib().sta_device_status(None), "status")
    assert got is out
    want, wlse, spread = kv_oracle.attention(q.double().numpy(), ref, table, lens, new, window)
    tol, eps = bounds(q.double().numpy(), ref, spread, want, lens, quant)
    x, y = got.double().cpu().numpy(), lse.double().cpu().numpy()
    for b in range(B):
        f = S if new is None else new[b]
        assert (x[b, :, f:] == 3.0).all()        # padding left as it was
        assert np.array_equal(np.isnan(x[b, :, :f]), np.isnan(want[b, :, :f]))
        with np.errstate(invalid="ignore"):
            bad = np.abs(x[b, :, :f] - want[b, :, :f]) > tol[b, :, :f]
            same = x[b, :, :f] == want[b, :, :f]         # infinities
        assert not (bad & ~same).any(), (b, np.argwhere(bad)[:4])
        nan = np.isnan(wlse[b, :, :f])
        assert np.array_equal(np.isnan(y[b, :, :f]), nan)
        gone = np.isneginf(wlse[b, :, :f])
        assert np.isneginf(y[b, :, :f][gone]).all()
        ok = ~gone & ~nan
        y_, w_ = y[b, :, :f][ok], wlse[b, :, :f][ok]
        assert (np.abs(y_ - w_) <= eps + 2.0 ** -22 * np.abs(w_)).all()
    return got


BLOCKS = [(64, 16), (64, 128), (128, 64), (128, 32)]


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("d,block", BLOCKS)
@pytest.mark.parametrize("heads", [(1, 1), (8, 2), (16, 1), (12, 4)], ids=str)
def test_single_tokens(d, block, quant, heads):
    lens = [1, 2, 15, 16, 17, 31, 33, 64, 127, 129, 300, 1000]
    check(np.random.default_rng(200), lens, None, 1, *heads, d, block, quant)


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 100, 129, 5000])
def test_windows(quant, window):
    check(np.random.default_rng(201), [1, 16, 40, 200, 513], None, 1, 4, 2, 128, 16, quant, window)
    check(np.random.default_rng(202), [3, 16, 40, 200, 513], [3, 2, 3, 1, 3], 3, 4, 2, 64, 64,
          quant, window)


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("S,heads", [(2, (4, 4)), (5, (8, 2)), (5, (32, 8)), (8, (8, 2)),
                                     (7, (24, 2)), (16, (4, 1)), (9, (16, 1))], ids=str)
def test_several_tokens(quant, S, heads):
    lens = [S, S + 1, 40, 200, 777]
    check(np.random.default_rng(203), lens, None, S, *heads, 128, 32, quant)
    check(np.random.default_rng(204), lens, [S, 1, 0, max(1, S // 2), S], S, *heads, 64, 16, quant,
          window=50)


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("S,heads,window", [(17, (4, 4), 0), (100, (8, 2), 0), (129, (4, 4), 0),
                                            (130, (8, 2), 40), (257, (16, 1), 300),
                                            (300, (2, 2), 1), (64, (12, 4), 129)], ids=str)
def test_pieces_of_prompts(quant, d, S, heads, window):
    check(np.random.default_rng(205), [S, 333 + S, S + 1], [S, S, 3], S, *heads, d, 64, quant,
          window)
    check(np.random.default_rng(206), [S], None, S, *heads, d, 16, quant, window)


@pytest.mark.parametrize("quant", [False, True])
def test_empty_places_and_rows_that_see_nothing(quant):
    # unused places of the batch: with new_lens 0, and without new_lens
    check(np.random.default_rng(207), [0, 40, 0], [0, 2, 0], 2, 4, 2, 64, 16, quant)
    check(np.random.default_rng(208), [0, 40, 0], None, 1, 4, 2, 64, 16, quant)
    # more new tokens than the sequence has: the first ones have no position
    check(np.random.default_rng(209), [3, 40], None, 5, 8, 2, 128, 64, quant)
    check(np.random.default_rng(210), [0, 0], None, 1, 4, 2, 64, 16, quant)
    check(np.random.default_rng(211), [3, 0, 150], None, 140, 4, 2, 128, 64, quant)


@pytest.mark.parametrize("layout", ["bhsd", "sliced"])
@pytest.mark.parametrize("S", [1, 6, 150])
def test_layouts(layout, S):
    check(np.random.default_rng(212), [150, 400], None, S, 6, 2, 128, 32, True, layout=layout)


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("S", [1, 150])
def test_large_scores(quant, S):
    # scores up to a few hundred: the running maximum moves, weights vanish
    check(np.random.default_rng(213), [700, 300], None, S, 4, 2, 128, 16, quant, q_std=20.0)


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("S", [1, 3, 40, 140])
def test_nonfinite_values_reach_only_the_rows_that_see_them(quant, S):
    def edit(t, ref, table):
        code = float("nan")
        for pos, hh, col in ((400 - S, 0, 5), (400 - S // 2 - 1, 1, 40), (250, 1, 63)):
            blk = int(table[0, pos // 32])
            t["v_cache"][blk, hh, pos % 32, col] = code
            ref["v"][blk, hh, pos % 32, col] = np.nan
    check(np.random.default_rng(214), [400], None, S, 4, 2, 64, 32, quant, edit=edit)


@pytest.mark.parametrize("S", [1, 40])
def test_infinite_values(S):
    def edit(t, ref, table):
        for pos, hh, col, x in ((399, 0, 5, np.inf), (400 - S, 1, 7, -np.inf), (10, 0, 9, np.inf)):
            blk = int(table[0, pos // 32])
            t["v_cache"][blk, hh, pos % 32, col] = x
            ref["v"][blk, hh, pos % 32, col] = x
    with np.errstate(invalid="ignore"):
        check(np.random.default_rng(215), [400], None, S, 4, 2, 64, 32, False, edit=edit)


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("S", [1, 3, 40, 140, 300])
def test_nan_keys_reach_the_rows_that_see_them(quant, S):
    # every place of a tile, first tokens and last ones, and the only token
    def edit(t, ref, table):
        for b, pos, hh in ((0, 400 - S, 0), (1, 403 - S // 2 - 1, 1), (2, 399, 0)):
            blk = int(table[b, pos // 32])
            t["k_cache"][blk, hh, pos % 32, 3] = float("nan")
            ref["k"][blk, hh, pos % 32, 3] = np.nan
        blk = int(table[3, 0])
        t["k_cache"][blk, :, 0, 9] = ref["k"][blk, :, 0, 9] = float("nan")
    with np.errstate(invalid="ignore"):
        check(np.random.default_rng(224), [400, 403, 400, 1], [S, S, S, 1], S, 4, 2, 64, 32, quant,
              edit=edit)


def test_e4m3_numbers_of_every_size():
    # all 254 finite numbers, the subnormal ones among them, under scales from
    # 2^-60 to 2^20: with one token each, the output is the token's value
    d, block, n = 128, 16, 4
    codes = torch.arange(256, dtype=torch.uint8)
    codes = codes[(codes & 127) != 127].repeat(3)[:n * d].view(n, 1, 1, d)
    vc = codes.view(torch.float8_e4m3fn).expand(n, 1, block, d).contiguous().cuda()
    kc = torch.zeros_like(vc.view(torch.uint8)).view(torch.float8_e4m3fn)
    vs = torch.tensor([[2.0 ** -60], [1.0], [2.0 ** 7], [2.0 ** 20]], device="cuda")
    for S in (1, 300):
        q = torch.ones((n, 1, S, d), dtype=torch.bfloat16, device="cuda")
        one = torch.ones(n, dtype=torch.int32, device="cuda")
        out = sta.kv_cache_attention(q, kc, vc, torch.arange(n, device="cuda").int()[:, None], one,
                                     k_scale=torch.ones_like(vs), v_scale=vs, new_lens=one)
        assert torch.equal(out[:, 0, 0].double(), vc[:, 0, 0].double() * vs.double())


def test_scales_far_apart():
    # blocks whose values differ by 2^40 and keys of every size
    def edit(t, ref, table):
        nb, h = t["v_scale"].shape
        rng = np.random.default_rng(1)
        f = torch.from_numpy(2.0 ** rng.integers(-40, 1, (nb, h))).float()
        t["v_scale"], ref["vs"] = t["v_scale"] * f, ref["vs"] * f.double().numpy()
        f = torch.from_numpy(2.0 ** rng.integers(-6, 1, (nb, h))).float()
        t["k_scale"], ref["ks"] = t["k_scale"] * f, ref["ks"] * f.double().numpy()
    for S in (1, 130):
        check(np.random.default_rng(216), [700], None, S, 4, 2, 128, 16, True, edit=edit)


def test_long_context_of_few_rows():
    check(np.random.default_rng(217), [40000, 20001], None, 1, 2, 1, 64, 128, True)
    check(np.random.default_rng(218), [30000], None, 2, 1, 1, 128, 16, False)


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("S,heads,most", [(1, (4, 4), 300), (2, (8, 2), 700), (3, (8, 1), 130),
                                          (12, (4, 2), 500), (20, (3, 1), 260),
                                          (70, (4, 1), 400)], ids=str)
def test_many_short_sequences(quant, S, heads, most):
    # hundreds of items of one tile to a few: a thread block has many of them, and
    # its first and last ones in part
    rng = np.random.default_rng(225)
    B = 24 if S == 70 else 90 if S > 3 else 260
    lens = [int(x) for x in rng.integers(0, most, B)]
    new = [int(min(n, rng.integers(0, S + 1))) for n in lens]
    check(rng, lens, new, S, *heads, 64, 16, quant)
    check(rng, lens, new, S, *heads, 128, 64, quant, window=90)


def test_uneven_lengths_move_the_division():
    # the same sequence among others of every length: its results differ by
    # where it is divided, within the bounds
    rng = np.random.default_rng(226)
    for n in (127, 128, 129, 1000, 20000):
        check(rng, [n, 5000, 1, 640], None, 1, 4, 1, 128, 32, True)


@pytest.mark.parametrize("S", [1, 140])
def test_cache_beyond_32_bit_offsets(S):
    # only the blocks in use are initialised
    d, block, nb, n = 128, 128, 140000, 300
    rng = np.random.default_rng(219)
    t, ref, table = kv_cases.rand_cache(rng, [n], 1, d, block, True, extra=0, junk=False)
    q = kv_cases.bf16(rng, (1, 4, S, d))
    kc, vc = (torch.empty((nb, 1, block, d), dtype=torch.float8_e4m3fn, device="cuda")
              for _ in range(2))
    ks, vs = (torch.empty((nb, 1), device="cuda") for _ in range(2))
    m = t["k_cache"].shape[0]
    kc[-m:], vc[-m:] = t["k_cache"].cuda(), t["v_cache"].cuda()
    ks[-m:], vs[-m:] = t["k_scale"].cuda(), t["v_scale"].cuda()
    out = sta.kv_cache_attention(q.cuda(), kc, vc, kv_cases.i32(table + nb - m), kv_cases.i32([n]),
                                 k_scale=ks, v_scale=vs)
    want, _, spread = kv_oracle.attention(q.double().numpy(), ref, table, [n], None, 0)
    tol, _ = bounds(q.double().numpy(), ref, spread, want, [n], True)
    assert (np.abs(out.double().cpu().numpy() - want) <= tol).all()
    # and storing there
    x = kv_cases.bf16(rng, (1, 1, 1, d))
    sta.kv_cache_append(x.cuda(), x.cuda(), kc, vc, kv_cases.i32([[nb - 1]]), kv_cases.i32([7]),
                        k_scale=ks, v_scale=vs)
    sc = float(vs[nb - 1, 0])
    assert np.array_equal(vc[nb - 1, 0, 6].double().cpu().numpy(),
                          kv_oracle.e4m3_round(x[0, 0, 0].double().numpy() / sc))


def test_bad_blocks_are_reported_and_skipped():
    rng = np.random.default_rng(220)
    for S in (1, 150):
        t, ref, table = kv_cases.rand_cache(rng, [200, 200], 2, 64, 16, True)
        q = kv_cases.bf16(rng, (2, 4, S, 64)).cuda()
        g = kv_cases.cuda(t)
        args = (g["k_cache"], g["v_cache"])
        kw = dict(k_scale=g["k_scale"], v_scale=g["v_scale"])
        good = sta.kv_cache_attention(q, *args, kv_cases.i32(table), kv_cases.i32([200] * 2), **kw)
        for bad in (-1, t["k_cache"].shape[0], 2 ** 31 - 1, -2 ** 31):
            broken = table.copy()
            broken[0, 3] = bad
            out = sta.kv_cache_attention(q, *args, kv_cases.i32(broken), kv_cases.i32([200] * 2),
                                         **kw)
            assert sta.lib().sta_device_status(None) == 6
            assert torch.equal(out[1], good[1])
        for n in (10 ** 6, 2 ** 31 - 1):
            out = sta.kv_cache_attention(q, *args, kv_cases.i32(table), kv_cases.i32([n, 200]),
                                         **kw)
            assert sta.lib().sta_device_status(None) == 6
        out = sta.kv_cache_attention(q, *args, kv_cases.i32(table), kv_cases.i32([-5, 200]), **kw)
        assert sta.lib().sta_device_status(None) == 0
        assert torch.equal(out[1], good[1]) and not out[0].any()


@pytest.mark.parametrize("S", [1, 5, 150])
def test_streams_and_repetition(S):
    # two calls at once on two streams, and the same call again: the same bits
    rng = np.random.default_rng(221)
    cases = []
    for lens in ([3000, 200, 900], [5000, 5000, 4]):
        new = [min(S, n) for n in lens]
        t, _, table = kv_cases.rand_cache(rng, lens, 2, 128, 32, True)
        g = kv_cases.cuda(t)
        q = kv_cases.bf16(rng, (3, 8, S, 128)).cuda()
        out = torch.zeros_like(q)
        cases.append((q, g["k_cache"], g["v_cache"], kv_cases.i32(table), kv_cases.i32(lens),
                      g["k_scale"], g["v_scale"], kv_cases.i32(new), 0, out))
    ref = [sta.kv_cache_attention(*c).clone() for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(5):
        for c, st in zip(cases, streams):
            c[-1].zero_()
            st.wait_stream(torch.cuda.current_stream())
        for c, st in zip(cases, streams):
            with torch.cuda.stream(st):
                sta.kv_cache_attention(*c)
        torch.cuda.synchronize()
        for c, r in zip(cases, ref):
            assert torch.equal(c[-1], r)


@pytest.mark.parametrize("S", [1, 4])
def test_step_of_a_model_in_a_graph(S):
    """Append and attention as a decoding loop runs them: captured once, the
    lengths advance on the device; every step equals the oracle's on the numbers
    that the cache then holds, and two graphs replayed in turn keep their own
    workspaces."""
    rng = np.random.default_rng(222)
    B, hq, hkv, d, block, steps = 2, 8, 2, 64, 16, 9
    lens0 = np.array([30, 5])
    t, _, table = kv_cases.rand_cache(rng, [80, 80], hkv, d, block, True, junk=False)
    g = kv_cases.cuda(t)
    tab = sta.rope_table(80, d)
    q, k, v = (torch.zeros((B, S, h, d), dtype=torch.bfloat16, device="cuda").transpose(1, 2)
               for h in (hq, hkv, hkv))
    n = kv_cases.i32(lens0)
    tb = kv_cases.i32(table)
    kw = dict(k_scale=g["k_scale"], v_scale=g["v_scale"])
    outs = [torch.zeros((B, hq, S, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    qr = torch.zeros_like(q)
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    with torch.cuda.graph(graphs[0]):
        n.add_(S)
        sta.kv_cache_append(k, v, g["k_cache"], g["v_cache"], tb, n, q=q, rope=tab, q_out=qr, **kw)
        sta.kv_cache_attention(qr, g["k_cache"], g["v_cache"], tb, n, out=outs[0], **kw)
    with torch.cuda.graph(graphs[1]):
        sta.kv_cache_attention(qr, g["k_cache"], g["v_cache"], tb, n, window=20, out=outs[1], **kw)
    lens = lens0.copy()
    for _ in range(steps):
        lens = lens + S
        for x in (q, k, v):
            x.copy_(kv_cases.bf16(rng, tuple(x.shape)))
        graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        ref = {"k": g["k_cache"].double().cpu().numpy(), "v": g["v_cache"].double().cpu().numpy(),
               "ks": g["k_scale"].double().cpu().numpy(),
               "vs": g["v_scale"].double().cpu().numpy()}
        qd = qr.double().cpu().numpy()
        for out, window in zip(outs, (0, 20)):
            want, _, spread = kv_oracle.attention(qd, ref, table, lens, None, window)
            tol, _ = bounds(qd, ref, spread, want, lens, True)
            assert (np.abs(out.double().cpu().numpy() - want) <= tol).all()


def test_prompt_through_the_cache_is_swa_forward():
    """A prompt attended as one piece over an unquantised cache, and in pieces,
    is the sliding-window attention that the library computes on plain tensors:
    both round the same scores' weights to bf16, each to within 2^-7 of the
    spread of the values and half a bf16 step of the result."""
    rng = np.random.default_rng(223)
    S, hq, hkv, d, block, window = 768, 8, 2, 128, 64, 200
    q, k, v = (kv_cases.bf16(rng, (1, h, S, d)).cuda() for h in (hq, hkv, hkv))
    want = sta.swa_forward(q, k, v, window).double()
    kc, vc, _, _ = sta.kv_cache_empty(S // block, hkv, block, d)
    table = kv_cases.i32(rng.permutation(S // block)[None])
    outs = torch.zeros_like(q)
    at = 0
    for n in (300, 1, 467):
        x = slice(at, at + n)
        at += n
        lens = kv_cases.i32([at])
        sta.kv_cache_append(k[:, :, x], v[:, :, x], kc, vc, table, lens)
        sta.kv_cache_attention(q[:, :, x], kc, vc, table, lens, window=window, out=outs[:, :, x])
    whole = sta.kv_cache_attention(q, kc, vc, table, lens, window=window)
    spread = sta.swa_forward(q, k, v.abs(), window).double()
    tol = 4 * (2.0 ** -8 + 2.0 ** -11) * spread * (1 + 2.0 ** -7) + 2 * 2.0 ** -8 * want.abs()
    for x in (outs, whole):
        assert ((x.double() - want).abs() <= tol).all()
