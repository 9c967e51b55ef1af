"""Paged cache, attention: inputs at the edges of what the kernels' number formats
and their exchange of maxima and sums hold.  Bounds as derived in
test_gpu_kv_attention.py."""
import numpy as np
import pytest
import torch

import block_sparse_local_b200 as sta
from oracle import kv_oracle
from tests import kv_cases
from tests.test_gpu_kv_attention import bounds

pytestmark = pytest.mark.gpu


def on_gpu(t, table, lens, q, new=None, window=0):
    """The call on the GPU, as a function that can be repeated."""
    g = kv_cases.cuda(t)
    args = (q.cuda(), g["k_cache"], g["v_cache"], kv_cases.i32(table), kv_cases.i32(lens))
    kw = dict(k_scale=g["k_scale"], v_scale=g["v_scale"], window=window, return_lse=True,
              new_lens=None if new is None else kv_cases.i32(new))
    return lambda: sta.kv_cache_attention(*args, **kw)


def status_ok():
    torch.cuda.synchronize()
    sta._check(sta.lib().sta_device_status(None), "status")


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("S,group", [(1, 8), (1, 16), (2, 16), (4, 16), (9, 16)], ids=str)
def test_scores_that_rise_to_the_last_tile(S, group, quant):
    """Key 128 i + t has 2 i in its first column and little elsewhere, and the
    queries are large: with q_0 > 0 a row's scores rise by q_0 i / 4 from tile to
    tile, so the reference rises with every tile, the last of an item among them,
    and what was summed up before is scaled.  160 items on 148 SMs, so most have
    all of their tiles in one thread block.  The right numbers, and always the same
    bits."""
    rng = np.random.default_rng(300 + S * group)
    B, hkv, d, block = 40, 4, 64, 64
    lens = [int(x) for x in rng.integers(1400, 1920, B)]
    lens[:3] = [1920, 1793, 1792]
    t, ref, table = kv_cases.rand_cache(rng, lens, hkv, d, block, quant)
    if quant:
        t["k_scale"].fill_(1.0), ref["ks"].fill(1.0)
    dtype = t["k_cache"].dtype
    for b, n in enumerate(lens):
        for i in range(-(-n // block)):
            blk, live = int(table[b, i]), min(block, n - i * block)
            x = torch.from_numpy(rng.standard_normal((hkv, live, d)) / 16).float()
            x[:, :, 0] = 2.0 * (i * block // 128)           # up to 28: exact in e4m3
            x = x.to(dtype)
            raw = torch.uint8 if quant else torch.int16
            t["k_cache"].view(raw)[blk, :, :live] = x.view(raw)
            ref["k"][blk, :, :live] = x.double().numpy()
    q = kv_cases.bf16(rng, (B, group * hkv, S, d), 20.0)
    call = on_gpu(t, table, lens, q)
    out, lse = call()
    status_ok()
    want, wlse, spread = kv_oracle.attention(q.double().numpy(), ref, table, lens, None, 0)
    tol, eps = bounds(q.double().numpy(), ref, spread, want, lens, quant)
    assert (np.abs(out.double().cpu().numpy() - want) <= tol).all()
    assert (np.abs(lse.double().cpu().numpy() - wlse) <= eps + 2.0 ** -22 * np.abs(wlse)).all()
    for _ in range(30):
        again, lse2 = call()
        assert torch.equal(again, out) and torch.equal(lse2, lse)
    status_ok()


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("S", [1, 5, 10, 20, 40, 300])
def test_queries_of_every_size(S, quant):
    """Queries times 2^e over keys times 2^-e have the same scores, and every
    product, sum and scale of the calculation is the same but for its exponent: the
    same bits, up to bf16's largest numbers.  (The keys of a bf16 cache stay normal
    numbers.)"""
    rng = np.random.default_rng(310)
    lens, d, block = [400, 1 + S, 77 + S], 64, 32
    t, ref, table = kv_cases.rand_cache(rng, lens, 2, d, block, quant, junk=False)
    q = kv_cases.bf16(rng, (3, 4, S, d)).clamp(-3.5, 3.5)
    q[q.abs() < 2.0 ** -8] = 0.0                 # times 2^-110 still a normal number
    out, lse = on_gpu(t, table, lens, q)()
    status_ok()
    want, _, spread = kv_oracle.attention(q.double().numpy(), ref, table, lens, None, 0)
    tol, _ = bounds(q.double().numpy(), ref, spread, want, lens, quant)
    assert (np.abs(out.double().cpu().numpy() - want) <= tol).all()
    for e in (-110, -101, -60, 60, 99, 101) + ((103, 113, 115, 120, 126) if quant else ()):
        qe = (q.double() * 2.0 ** e).to(torch.bfloat16)
        assert torch.isfinite(qe).all() and torch.equal(qe.double(), q.double() * 2.0 ** e)
        te = dict(t)
        name = "k_scale" if quant else "k_cache"
        te[name] = (t[name].double() * 2.0 ** -e).to(t[name].dtype)
        o, l = on_gpu(te, table, lens, qe)()
        status_ok()
        assert torch.equal(o, out), e
        assert torch.equal(l, lse), e


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("S", [1, 5, 10, 20, 40, 300])
@pytest.mark.parametrize("what", ["inf", "-inf", "nan"])
def test_nonfinite_queries_make_their_row_nan(what, S, quant):
    """Infinity times a key is infinite or NaN, so such a row's softmax is NaN, also
    where all its scores are -inf.  Rows that see nothing stay 0; the others do not
    notice.  The last sequence has one token, the one before none for its first
    rows."""
    rng = np.random.default_rng(311)
    lens, new, d, block = [400, 77 + S, S, 1], [S, S, S, 1], 64, 32
    lens[2] = max(1, S - 2)
    t, ref, table = kv_cases.rand_cache(rng, lens, 2, d, block, quant)
    q = kv_cases.bf16(rng, (4, 4, S, d))
    finite = q.clone()
    x = float(what)
    for b, h, s, c in ((0, 1, 0, 3), (0, 2, S - 1, 60), (1, 0, S // 2, 0), (2, 3, 0, 9),
                       (2, 0, S - 1, 9), (3, 0, 0, 5), (3, 1, 0, 63), (3, 2, 0, 31), (3, 3, 0, 1)):
        q[b, h, s, c] = x
    out, lse = on_gpu(t, table, lens, q, new)()
    status_ok()
    with np.errstate(invalid="ignore"):
        want, wlse, spread = kv_oracle.attention(q.double().numpy(), ref, table, lens, new, 0)
    tol, eps = bounds(finite.double().numpy(), ref, spread, want, lens, quant)
    got, glse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    nans = 0
    for b in range(4):
        f = new[b]
        w, g = want[b, :, :f], got[b, :, :f]
        # a non-finite query spoils its whole row
        row = np.isnan(w).any(-1, keepdims=True) & np.ones(w.shape, dtype=bool)
        nans += row.sum() // d
        assert np.array_equal(np.isnan(g), row), (b, np.argwhere(np.isnan(g) != row)[:4])
        assert (np.abs(g - w) <= tol[b, :, :f])[~row].all()
        wl, gl = wlse[b, :, :f], glse[b, :, :f]
        assert np.array_equal(np.isnan(gl), row[..., 0])
        gone = np.isneginf(wl)
        assert np.isneginf(gl[gone]).all()
        ok = ~gone & ~row[..., 0]
        assert (np.abs(gl[ok] - wl[ok]) <= eps + 2.0 ** -22 * np.abs(wl[ok])).all()
    assert nans >= 7


@pytest.mark.parametrize("window", [0, 100])
@pytest.mark.parametrize("block", [16, 64])
@pytest.mark.parametrize("S", [1, 5, 10, 20, 40, 300])
def test_zero_queries_and_zero_keys(S, block, window):
    """Rows of zeros over blocks of zeros, whose scale is the smallest that appending
    leaves, or 0 as in an empty cache: the scores are 0 and the weights equal.  The
    product of both scales is below fp32's range; masked places stay masked."""
    rng = np.random.default_rng(320)
    lens, d = [400, 77 + S, S, 130 + S], 64
    t, ref, table = kv_cases.rand_cache(rng, lens, 2, d, block, True)
    raw = t["k_cache"].view(torch.uint8)
    for b, n in enumerate(lens):
        for i in range(-(-n // block)):
            blk, kind = int(table[b, i]), int(rng.integers(0, 3)) if b < 3 else 1
            if kind == 0:                                   # some blocks as they were
                continue
            live = min(block, n - i * block)
            raw[blk, :, :live] = 0
            ref["k"][blk, :, :live] = 0.0
            t["k_scale"][blk] = ref["ks"][blk] = 2.0 ** -64 if kind == 1 else 0.0
    q = kv_cases.bf16(rng, (4, 4, S, d))
    q[:, :2] = 0.0
    q[:, 3, ::2] = 0.0
    out, lse = on_gpu(t, table, lens, q, None, window)()
    status_ok()
    want, wlse, spread = kv_oracle.attention(q.double().numpy(), ref, table, lens, None, window)
    tol, eps = bounds(q.double().numpy(), ref, spread, want, lens, True)
    assert (np.abs(out.double().cpu().numpy() - want) <= tol).all()
    assert (np.abs(lse.double().cpu().numpy() - wlse) <= eps + 2.0 ** -22 * np.abs(wlse)).all()
