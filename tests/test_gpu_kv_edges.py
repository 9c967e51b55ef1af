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
