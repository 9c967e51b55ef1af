"""Random paged caches for the key/value cache tests, as tensors and as the
oracle's float64 view of the same numbers."""
import numpy as np
import torch


def rand_cache(rng, lens, hkv, d, block, quantised, extra=2, junk=True):
    """Blocks in random order, something in every slot; slots behind a sequence's
    end (and unused blocks) hold NaN and the largest numbers when junk."""
    per = [-(-n // block) for n in lens]
    nb, width = sum(per) + extra, max(max(per), 1)
    order = rng.permutation(nb)
    table = np.full((len(lens), width), -7 if junk else 0, dtype=np.int32)   # not to be read
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = order[at:at + n]
        at += n
    size = np.exp(0.4 * rng.standard_normal((1, hkv, 1, d)))
    t, ref = {}, {}
    for name in ("k", "v"):
        x = torch.from_numpy(rng.standard_normal((nb, hkv, block, d)) * size).float()
        if quantised:
            amax = x.abs().amax(dim=(2, 3)).double()
            scale = torch.exp2(torch.ceil(torch.log2(amax / 448.0))).float()
            # blocks differ by powers of two, so that the scales matter
            x = (x / scale[:, :, None, None]).to(torch.float8_e4m3fn)
            scale = scale * torch.from_numpy(2.0 ** rng.integers(-2, 2, (nb, hkv))).float()
            t[name + "_scale"] = scale
        else:
            x = x.to(torch.bfloat16)
            scale = torch.ones((nb, hkv))
            t[name + "_scale"] = None
        ref[name] = x.double().numpy()
        ref[name + "s"] = scale.double().numpy()
        if junk:
            used = np.zeros((nb, block), dtype=bool)
            for b, n in enumerate(lens):
                for i in range(per[b]):
                    used[table[b, i], :max(0, min(block, n - i * block))] = True
            un = torch.from_numpy(~used)[:, None, :, None].expand(x.shape)
            bad = torch.tensor([float("nan"), 448.0, -448.0, float("nan")]).to(x.dtype)
            raw = x.view(torch.uint8 if quantised else torch.int16)
            fill = bad.view(raw.dtype)[torch.from_numpy(rng.integers(0, 4, x.shape))]
            x = torch.where(un, fill, raw).view(x.dtype)
        t[name + "_cache"] = x
    return t, ref, table


def bf16(rng, shape, std=1.0):
    return torch.from_numpy(rng.standard_normal(shape) * std).to(torch.bfloat16)


def cuda(t):
    return {k: (x.cuda() if x is not None else None) for k, x in t.items()}


def i32(x, device="cuda"):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=device)
