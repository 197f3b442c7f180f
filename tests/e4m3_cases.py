"""Inputs and layouts shared by the tests of the 8-bit cache."""
import numpy as np
import torch

import oracle.cache_e4m3 as ref
import workloads as W


def codes_to_f64(t):
    return t.detach().cpu().float().numpy().astype(np.float64)


def empty_cache(nb, h_kv, d, fill=0):
    """Code and exponent tensors on the GPU, every byte `fill`."""
    c = torch.full((nb, h_kv, 16, d), fill, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    e = torch.full((nb, h_kv, 16), fill, dtype=torch.uint8, device="cuda")
    return c, c.clone(), e, e.clone()


def cache_from(x):
    """Quantised cache (CPU tensors: codes float8, exponents uint8) of values
    x [nb, h_kv, 16, d], through the oracle."""
    codes, e = ref.quantise_ref(x)
    c8 = torch.from_numpy(codes).float().to(torch.float8_e4m3fn)  # exact: codes are e4m3 numbers
    return c8, torch.from_numpy(e)


def values(c8, e):
    """Stored values in float64, [nb, 16, h_kv, d] (the bf16 caches' order)."""
    v = ref.values_ref(codes_to_f64(c8), e.cpu().numpy())
    return np.ascontiguousarray(v.transpose(0, 2, 1, 3))


def token_slots(cu, lens, table, total):
    """(page, slot) of every packed token, None where it has none."""
    out = [None] * total
    for b, n in enumerate(lens):
        for t in range(cu[b], cu[b + 1]):
            if t < total:
                pos = n - cu[b + 1] + t
                out[t] = (int(table[b, pos // 16]), pos % 16)
    return out


def decode_case(B_lens, h_kv, g, d, seed, v_mult=1.0):
    """q, quantised caches, table and lengths of a decode batch (CPU)."""
    table, nb = W.paged_layout(B_lens, seed)
    q = W.normal((len(B_lens), h_kv * g, d), seed * 5 + 1, torch.bfloat16)
    k = W.normal((nb, h_kv, 16, d), seed * 5 + 2, torch.bfloat16)
    v = W.normal((nb, h_kv, 16, d), seed * 5 + 3, torch.bfloat16, mult=v_mult)
    kc, ks = cache_from(k.double().numpy())
    vc, vs = cache_from(v.double().numpy())
    return q, kc, vc, ks, vs, table, torch.tensor(B_lens, dtype=torch.int32)
