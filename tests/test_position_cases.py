"""That position_cases.py finds what it is for: mistakes planted in the oracle's inputs,
on the CPU, one page each, move the result past the bound."""
import numpy as np
import pytest
import torch

import position_cases as PC
from test_gpu_decode_e4m3 import reference as reference8
from test_gpu_decode_shared import reference


def outside(O, wrong):
    return (np.abs(wrong - O) > PC.BOUND * O).any()


@pytest.mark.parametrize("i", range(len(PC.SHARED)))
def test_shared(i):
    args = PC.shared_case(*PC.SHARED[i], seed=71 + i)
    row = [int(torch.argmax(args[6]))]
    O = reference(*args, rows=row)[0][row]
    v, ptab, tab = args[2], args[3], args[5]
    P, n = (int(args[4]) + 15) // 16, (int(args[6][row[0]]) + 15) // 16
    for pages, count in ((ptab, P), (tab[row[0]], n)):
        for at in {0, count // 2, count - 1} if count else ():
            for factor in (0.0, 2.0):  # a page lost, counted twice
                bad = v.clone()
                bad[int(pages[at])] *= factor
                assert outside(O, reference(args[0], args[1], bad, *args[3:], rows=row)[0][row])


@pytest.mark.parametrize("i", range(len(PC.E4M3)))
def test_e4m3(i):
    q, kc, vc, ks, vs, table, n = PC.e4m3_case(*PC.E4M3[i], seed=81 + i)
    b = int(torch.argmax(n))
    one = lambda t: t[b:b + 1]
    O = reference8(one(q), kc, vc, ks, vs, one(table), one(n))[0]
    count = (int(n[b]) + 15) // 16
    for at in (0, count // 2, count - 1):
        bad = vc.clone()
        bad.view(torch.uint8)[int(table[b, at])] = 0
        assert outside(O, reference8(one(q), kc, bad, ks, vs, one(table), one(n))[0])
