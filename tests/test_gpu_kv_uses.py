"""Paged cache, attention and appending: uses that the documentation allows beside
the ordinary ones.  Bounds as derived in test_gpu_kv_attention.py."""
import numpy as np
import pytest
import torch

import block_sparse_local_b200 as sta
from oracle import kv_oracle
from tests import kv_cases
from tests.test_gpu_kv_attention import bounds, check
from tests.test_gpu_kv_edges import status_ok

pytestmark = pytest.mark.gpu
I32 = kv_cases.i32


def _close(out, q, ref, table, lens, new, window, quant):
    qd = q.double().cpu().numpy()
    want, _, spread = kv_oracle.attention(qd, ref, table, lens, new, window)
    tol, _ = bounds(qd, ref, spread, want, lens, quant)
    got = out.double().cpu().numpy()
    for b in range(len(lens)):
        f = qd.shape[2] if new is None else new[b]
        assert (np.abs(got[b, :, :f] - want[b, :, :f]) <= tol[b, :, :f]).all(), b


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("B,S,heads", [(1500, 1, (4, 1)), (900, 2, (16, 1)), (700, 34, (2, 1))],
                         ids=str)
def test_more_sequences_than_threads(B, S, heads, quant):
    # a thread of the division has several sequences, empty ones among them
    rng = np.random.default_rng(400)
    lens = [int(x) if x > 30 else 0 for x in rng.integers(0, 300, B)]
    new = [int(min(n, rng.integers(0, S + 1))) for n in lens]
    check(rng, lens, new, S, *heads, 64, 16, quant)


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("S,heads", [(1, (128, 1)), (1, (72, 1)), (3, (43, 1)), (2, (32, 1)),
                                     (1, (65, 1)), (33, (2, 1))], ids=str)
def test_rows_around_the_forms_borders(S, heads, quant):
    check(np.random.default_rng(401), [300, 1 + S, 1000], None, S, *heads, 128, 32, quant)


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("S", [1, 6, 40, 300])
def test_blocks_in_front_of_the_window_are_given_back(S, quant):
    # their entries are not read
    rng = np.random.default_rng(402)
    lens, block, window = [900, 333 + S, 1200], 16, 70
    t, ref, table = kv_cases.rand_cache(rng, lens, 2, 64, block, quant)
    q = kv_cases.bf16(rng, (3, 4, S, 64)).cuda()
    freed = table.copy()
    for b, n in enumerate(lens):
        freed[b, :max(0, n - S - window + 1) // block] = -1
    assert (freed[0] == -1).sum() > 20
    g = kv_cases.cuda(t)
    out = sta.kv_cache_attention(q, g["k_cache"], g["v_cache"], I32(freed), I32(lens),
                                 k_scale=g["k_scale"], v_scale=g["v_scale"], window=window)
    status_ok()
    _close(out, q, ref, table, lens, None, window, quant)


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("S", [1, 5, 40, 150])
def test_caches_with_heads_outermost_and_shared_blocks(S, quant):
    # [heads][blocks] for K, [blocks][K or V][heads] with room between for V; two
    # sequences have their first blocks in common, one has a block twice
    rng = np.random.default_rng(403)
    lens, block, d, H = [200, 180 + S, 97 + S], 16, 128, 3
    t, ref, table = kv_cases.rand_cache(rng, lens, H, d, block, quant, junk=False)
    table[1, :5] = table[0, :5]
    table[2, 3] = table[2, 0]
    g = kv_cases.cuda(t)
    nb = g["k_cache"].shape[0]
    raw = torch.uint8 if quant else torch.int16
    dt = g["k_cache"].dtype
    kc = torch.zeros((H, nb, block, d), dtype=raw, device="cuda").view(dt).transpose(0, 1)
    vc = torch.zeros((nb, 2, H + 1, block, d), dtype=raw, device="cuda").view(dt)[:, 1, 1:]
    kc.view(raw).copy_(g["k_cache"].view(raw))
    vc.view(raw).copy_(g["v_cache"].view(raw))
    q = kv_cases.bf16(rng, (3, 2 * H, S, d)).cuda()
    # the batch innermost in the output
    out = torch.zeros((S, 2 * H, 3, d), dtype=torch.bfloat16, device="cuda").permute(2, 1, 0, 3)
    sta.kv_cache_attention(q, kc, vc, I32(table), I32(lens), k_scale=g["k_scale"],
                           v_scale=g["v_scale"], out=out)
    status_ok()
    _close(out, q, ref, table, lens, None, 0, quant)
    # appending there: the same numbers as in an ordinary cache
    x = kv_cases.bf16(rng, (3, H, 1, d)).cuda()
    at, own = I32([n + 1 for n in (lens[0], 3, 5)]), I32([[0] * 12 + [1], [2] * 13, [3] * 13])
    for a, b in ((kc, vc), (g["k_cache"], g["v_cache"])):
        ks, vs = ((None, None) if not quant else (g["k_scale"].clone(), g["v_scale"].clone()))
        sta.kv_cache_append(x, x, a, b, own, at, k_scale=ks, v_scale=vs)
    status_ok()
    assert torch.equal(kc.contiguous().view(raw), g["k_cache"].view(raw))
    assert torch.equal(vc.contiguous().view(raw), g["v_cache"].view(raw))


@pytest.mark.parametrize("quant", [False, True])
def test_inputs_that_repeat_themselves(quant):
    # expanded tensors: one token's keys for all heads, one query for the batch
    rng = np.random.default_rng(404)
    B, H, S, d, block = 2, 4, 3, 64, 16
    k, v = (kv_cases.bf16(rng, (B, 1, S, d)).cuda().expand(B, H, S, d) for _ in range(2))
    q = kv_cases.bf16(rng, (1, 8, S, d)).cuda().expand(B, 8, S, d)
    rope, table, lens = sta.rope_table(64, d), I32([[1, 0, 2, 3], [5, 4, 6, 7]]), I32([20, 9])
    got, want = [], []
    for res, f in ((got, lambda x: x), (want, lambda x: x.contiguous())):
        kc, vc, ks, vs = sta.kv_cache_empty(
            8, H, block, d, dtype=torch.float8_e4m3fn if quant else torch.bfloat16)
        qr = sta.kv_cache_append(f(k), f(v), kc, vc, table, lens, k_scale=ks, v_scale=vs, q=f(q),
                                 rope=rope)
        new = I32([S, S])
        out = sta.kv_cache_attention(f(q), kc, vc, table, lens, k_scale=ks, v_scale=vs,
                                     new_lens=new, window=2)
        res += [kc.view(torch.uint8 if quant else torch.int16), qr, out[:, :, 1:]]
    status_ok()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("S", [1, 20, 150])
def test_two_graphs_replayed_at_once(S):
    rng = np.random.default_rng(405)
    runs, streams = [], [torch.cuda.Stream() for _ in range(2)]
    for lens in ([4000, 900], [2500, 2500]):
        t, _, table = kv_cases.rand_cache(rng, lens, 2, 128, 64, True)
        g = kv_cases.cuda(t)
        q = kv_cases.bf16(rng, (2, 8, S, 128)).cuda()
        args = (q, g["k_cache"], g["v_cache"], I32(table), I32(lens), g["k_scale"], g["v_scale"])
        want = sta.kv_cache_attention(*args)
        out = torch.zeros_like(q)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            sta.kv_cache_attention(*args, out=out)
        runs.append((graph, out, want, args))
    for _ in range(20):
        for (graph, out, _, _), st in zip(runs, streams):
            out.zero_()
            st.wait_stream(torch.cuda.current_stream())
        for (graph, _, _, _), st in zip(runs, streams):
            with torch.cuda.stream(st):
                graph.replay()
        torch.cuda.synchronize()
        for _, out, want, _ in runs:
            assert torch.equal(out, want)
    status_ok()


def test_one_block_and_one_head_of_a_larger_cache():
    # the strides of dimensions of one are whatever the slice has
    rng = np.random.default_rng(406)
    d, block = 64, 16
    big = torch.zeros((5, 3, block, d), dtype=torch.bfloat16, device="cuda")
    kc, vc = big[2:3, 1:2], big[4:5, 2:3]
    x, y = (kv_cases.bf16(rng, (1, 1, 9, d)) for _ in range(2))
    sta.kv_cache_append(x.cuda(), y.cuda(), kc, vc, I32([[0]]), I32([9]))
    out = sta.kv_cache_attention(x.cuda()[:, :, :1], kc, vc, I32([[0]]), I32([1]))
    status_ok()
    assert torch.equal(out.cpu()[0, 0, 0], y[0, 0, 0])
    assert big.count_nonzero() == x.count_nonzero() + y.count_nonzero()
