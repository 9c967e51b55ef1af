"""Paged key/value cache on the CPU: the oracle's own pins, and the refusals of
the C entry points and of the Python calls (no kernel is launched)."""
import ctypes

import numpy as np
import pytest
import torch

import block_sparse_local_b200 as sta
from block_sparse_local_b200 import build as sta_build
from oracle import kv_oracle, swa_oracle


@pytest.fixture(scope="module")
def L():
    sta_build.build()
    return sta.lib()


# ------------------------------------------------------------------ oracle pins
def test_e4m3_rounding_agrees_with_torch_on_every_number_and_between():
    tab = kv_oracle.e4m3_table()
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(tab, codes, equal_nan=True)
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.uniform(-448, 448, 20000), rng.standard_normal(20000) * 1e-2,
                        (kv_oracle._POS[:-1] + kv_oracle._POS[1:]) / 2])
    x = x.astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(kv_oracle.e4m3_round(x.astype(np.float64)), want)
    assert kv_oracle.e4m3_round(np.array([1e9, -np.inf])).tolist() == [448.0, -448.0]
    assert np.isnan(kv_oracle.e4m3_round(np.array([np.nan]))).all()


def test_scale_is_the_smallest_power_of_two():
    for a, s in ((448.0, 1.0), (448.0001, 2.0), (447.0, 1.0), (224.0, 0.5), (0.0, 2.0 ** -64),
                 (1e-30, 2.0 ** -64), (1.75, 2.0 ** -8), (1.7501, 2.0 ** -7)):
        assert kv_oracle.e4m3_scale(a) == s


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_norms_and_relative_angles(interleaved):
    rng = np.random.default_rng(1)
    d = 64
    t = sta.rope_table(300, d, device="cpu").double().numpy()
    a, b = rng.standard_normal((2, d))
    dots = [kv_oracle.rotate(a, p + 17, t, interleaved) @ kv_oracle.rotate(b, p, t, interleaved)
            for p in (0, 5, 250)]
    assert np.allclose(dots, dots[0], atol=1e-5)
    assert np.allclose(kv_oracle.rotate(a, 0, t, interleaved), a)


def test_rope_table_far_positions():
    t = sta.rope_table(1000001, 64, device="cpu")
    ang = 1000000 * 10000.0 ** (-np.arange(0, 64, 2) / 64)
    assert np.allclose(t[1000000, :32].numpy(), np.cos(ang), atol=1e-6)
    assert np.allclose(t[1000000, 32:].numpy(), np.sin(ang), atol=1e-6)


def test_cache_attention_oracle_is_the_sliding_window_oracle():
    # all tokens new, blocks out of order: the same numbers as on plain tensors
    rng = np.random.default_rng(2)
    S, d, hq, hkv, block, window = 70, 8, 4, 2, 16, 23
    q, k, v = (rng.standard_normal((1, h, S, d)) for h in (hq, hkv, hkv))
    cache = {n: np.zeros((6, hkv, block, d)) for n in ("k", "v")}
    cache.update({n: np.ones((6, hkv)) for n in ("ks", "vs")})
    table = np.array([[3, 0, 5, 1, 4]])
    kv_oracle.append(cache, k, v, table, [S], None, None, False, False)
    out, lse, _ = kv_oracle.attention(q, cache, table, [S], None, window)
    want = swa_oracle.swa_forward(q[0], k[0], v[0], window)
    for h in range(hq):
        assert np.allclose(out[0, h], want[h][0]) and np.allclose(lse[0, h], want[h][1])


def test_append_oracle_token_by_token_equals_at_once():
    # power-of-two scales: moving a block's numbers to a larger scale loses
    # nothing in the normal range, so the order of arrival does not matter
    rng = np.random.default_rng(3)
    S, d, block = 40, 8, 16
    k, v = (rng.choice([-1, 1], (1, 1, S, d)) * rng.uniform(0.5, 2.0, (1, 1, S, d)) *
            2.0 ** rng.integers(0, 5, (1, 1, S, 1)) for _ in range(2))

    def empty():
        c = {n: np.zeros((3, 1, block, d)) for n in ("k", "v")}
        c.update({n: np.zeros((3, 1)) for n in ("ks", "vs")})
        return c

    table, a, b = np.array([[2, 0, 1]]), empty(), empty()
    kv_oracle.append(a, k, v, table, [S], None, None, False, True)
    for s in range(S):
        kv_oracle.append(b, k[:, :, s:s + 1], v[:, :, s:s + 1], table, [s + 1], None, None, False,
                         True)
    for n in a:
        assert np.array_equal(a[n], b[n])


# ------------------------------------------------------------------ refusals, C
P = [ctypes.c_void_p((i + 1) << 20) for i in range(16)]     # never dereferenced


def _i64(*x):
    return (ctypes.c_int64 * len(x))(*x)


def _append(L, **kw):
    a = dict(k=P[0], v=P[1], q=P[2], q_out=P[3], st=_i64(*[1 << 20, 1 << 14, 128] * 4), kc=P[4],
             vc=P[5], ks=P[6], vs=P[7], cst=_i64(1 << 16, 64 * 128, 1 << 16, 64 * 128), table=P[8],
             width=8, lens=P[9], new=None, rope=P[10], rows=512, inter=0, B=2, S=3, hq=8, hkv=8,
             d=128, nb=20, block=64, type=1)
    a.update(kw)
    return L.sta_kv_append(*a.values(), None)


def _attend(L, **kw):
    a = dict(q=P[0], out=P[1], lse=None, st=_i64(*[1 << 20, 1 << 14, 128] * 2), kc=P[4], vc=P[5],
             ks=P[6], vs=P[7], cst=_i64(1 << 16, 64 * 128, 1 << 16, 64 * 128), table=P[8], width=8,
             lens=P[9], new=None, window=0, ws=P[11], wsb=1 << 30, B=2, S=3, hq=8, hkv=8, d=128,
             nb=20, block=64, type=1)
    a.update(kw)
    return L.sta_kv_attention(*a.values(), None)


OFF8 = ctypes.c_void_p((1 << 20) + 8)
OFF2 = ctypes.c_void_p((1 << 20) + 2)
SHARED_BAD = [
    dict(kc=None), dict(vc=None), dict(table=None), dict(lens=None), dict(cst=None),
    dict(st=None), dict(kc=OFF8), dict(vc=P[4]), dict(table=OFF2), dict(lens=OFF2),
    dict(new=OFF2), dict(ks=OFF2), dict(B=0), dict(S=0), dict(hq=0), dict(hkv=0), dict(hkv=3),
    dict(nb=0), dict(width=0), dict(block=0), dict(type=2), dict(type=-1),
    dict(type=0), dict(ks=None), dict(vs=None), dict(vs=P[6]),
    dict(cst=_i64(64, 64 * 128, 1 << 16, 64 * 128)),           # blocks overlap
    dict(cst=_i64(1 << 16, 64 * 128 + 8, 1 << 16, 64 * 128)),  # rows not 16-byte aligned
    dict(width=1 << 25), dict(B=1 << 20, S=1 << 10),
]


@pytest.mark.parametrize("bad", SHARED_BAD + [
    dict(k=None), dict(v=None), dict(k=OFF8), dict(q_out=None), dict(q=None), dict(rope=None),
    dict(rope=OFF8), dict(rows=511), dict(inter=2), dict(q_out=P[0]), dict(q_out=P[4]),
    dict(st=_i64(*[1 << 20, 1 << 14, 129] * 4)), dict(st=_i64(*[1 << 20, -128, 128] * 4)),
    dict(st=_i64(*[1 << 20, 1 << 14, 128] * 3, 1 << 20, 0, 128)),          # rows of q_out overlap
    dict(q_out=P[2], st=_i64(*[1 << 20, 1 << 14, 128] * 3, 1 << 20, 1 << 15, 128)),
], ids=str)
def test_append_refuses(L, bad):
    assert _append(L, **bad) == 1


@pytest.mark.parametrize("bad", SHARED_BAD + [
    dict(q=None), dict(out=None), dict(q=OFF8), dict(out=P[0]), dict(out=P[5]), dict(lse=OFF2),
    dict(window=-1), dict(ws=None), dict(ws=OFF8), dict(wsb=1000),
    dict(st=_i64(*[1 << 20, 1 << 14, 129] * 2)),
    dict(st=_i64(*[1 << 20, 1 << 14, 128], 1 << 20, 0, 128)),
], ids=str)
def test_attention_refuses(L, bad):
    assert _attend(L, **bad) == 1


@pytest.mark.parametrize("call", [_append, _attend])
@pytest.mark.parametrize("bad", [dict(d=96), dict(d=256), dict(block=48), dict(block=256),
                                 dict(block=8)], ids=str)
def test_unsupported_sizes(L, call, bad):
    kw = dict(cst=_i64(1 << 20, 1 << 16, 1 << 20, 1 << 16), rows=4096, **bad)
    if call is _attend:
        kw.pop("rows")
    assert call(L, **kw) == 2


def test_workspace_size(L):
    f = L.sta_kv_attention_workspace
    assert f(0, 8, 8, 128) == -1 and f(1, 8, 3, 128) == -1 and f(1, 8, 8, 96) == -1
    assert 0 < f(1, 8, 8, 64) < f(1, 8, 8, 128) < 64 << 20
    assert f(1 << 20, 64, 1, 128) > 0


# ------------------------------------------------------------------ refusals, Python
def _args(dtype=torch.float8_e4m3fn, **kw):
    kc, vc, ks, vs = sta.kv_cache_empty(6, 2, 16, 64, dtype=dtype, device="cpu")
    a = dict(k_cache=kc, v_cache=vc, block_table=torch.zeros((1, 4), dtype=torch.int32),
             seq_lens=torch.ones(1, dtype=torch.int32), k_scale=ks, v_scale=vs)
    a.update(kw)
    return a


TOK = torch.zeros((1, 2, 3, 64), dtype=torch.bfloat16)


@pytest.mark.parametrize("kw", [
    dict(),                                                   # CPU tensors
    dict(k_cache=torch.zeros((6, 2, 16, 64), dtype=torch.float16)),
    dict(k_cache=torch.zeros((6, 2, 64, 16), dtype=torch.float8_e4m3fn).transpose(2, 3)),
    dict(k_scale=None), dict(k_scale=torch.zeros((6, 3))),
    dict(k_scale=torch.zeros((6, 2), dtype=torch.float64)),
    dict(block_table=torch.zeros((1, 4), dtype=torch.int64)),
    dict(block_table=torch.zeros((2, 4), dtype=torch.int32)),
    dict(seq_lens=torch.ones(2, dtype=torch.int32)),
    dict(new_lens=torch.ones(1, dtype=torch.int64)),
    dict(q=TOK.float()), dict(q=TOK.transpose(2, 3)), dict(q=TOK[..., :32]), dict(q=TOK[0]),
    dict(out=TOK[:, :1]), dict(window=-1),
    dict(q=torch.zeros((1, 3, 3, 64), dtype=torch.bfloat16)),
], ids=lambda k: ",".join(k))
def test_python_attention_refuses(kw):
    a = _args(**{"q": TOK, **kw})
    with pytest.raises(ValueError):
        sta.kv_cache_attention(**a)


@pytest.mark.parametrize("kw", [
    dict(), dict(v=TOK[:, :1]), dict(q=TOK), dict(q_out=TOK), dict(k=TOK.float(), v=TOK.float()),
    dict(q=TOK, rope=torch.zeros((63, 64))), dict(rope=torch.zeros((64, 32))),
    dict(rope=torch.zeros((64, 64), dtype=torch.float64)),
    dict(k=TOK[:, :1], v=TOK[:, :1]),
    dict(q=TOK, q_out=TOK[:, :1], rope=torch.zeros((64, 64))),
], ids=lambda k: ",".join(k))
def test_python_append_refuses(kw):
    a = _args(**{"k": TOK, "v": TOK, **kw})
    with pytest.raises(ValueError):
        sta.kv_cache_append(**a)


def test_empty_cache():
    k, v, ks, vs = sta.kv_cache_empty(3, 2, 16, 64, device="cpu")
    assert k.shape == (3, 2, 16, 64) and k.dtype == torch.bfloat16 and ks is None and vs is None
    with pytest.raises(ValueError):
        sta.kv_cache_empty(3, 2, 16, 64, dtype=torch.float16, device="cpu")
