"""Small weights of the 8-bit attention, seen by themselves: a first key takes most of the
weight and has a value in dimension 0 alone, n others of one small weight have theirs in
dimension 1.

What they add to dimension 1 is n w, off by n (2^-10 w + A): a half's rounding and that of
its third part (2^-11 of the weight's power of two each), and A where halves and e5m2 end:
(2^-25 + 2^-17 / 128) / 2 of the first key's weight, which is kept at more than 2: 1.5 *
2^-25 (all values have one scale).  Scores of one term are off by four roundings, 2^-22 of
at most 32, which moves weight and sum by less than 2^-15; exp2, the sums of n terms and the
division 2^-21 + 2 n 2^-24; and half a bf16 step is 2^-8 of the result."""
import math

import numpy as np
import pytest

from gpu_common import torch_cuda
from test_gpu_paged8 import Case8

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [1.0, 9.6, 14.2, 16.3, 17.0, 18.7, 20.0, 20.6, 22.2, 23.5, 24.0, 24.9])
@pytest.mark.parametrize("heads,new", [((4, 1, 128), 1), ((8, 2, 64), 4), ((64, 1, 128), 1)])
@pytest.mark.parametrize("n", [127, 900, 20000])
def test_small_weights_beside_a_large_one(n, heads, new, bits):
    torch = torch_cuda()
    hq, hkv, hd = heads
    c = Case8([n + 1], [new], hq, hkv, hd, seed=41, spread=0)
    c.q[:] = 0.0
    c.q[:, :, 0] = bits * math.log(2.0) * hd ** 0.5 / 128    # (the key's 128 is a code, and stays as it is)
    c.d["q"] = c.q.cuda()
    c.k[0][:] = 0.0
    c.k[0][0, :, 0] = 128.0
    c.v[0][:] = 0.0
    c.v[0][0, :, 0] = 1.0
    c.v[0][1:, :, 1] = 1.0
    c.place(0, torch.arange(n + 1))
    c.upload()
    s = float(c.q[0, 0, 0]) * 128 * hd ** -0.5
    got = c.run().double().cpu().numpy()[:new]
    for j in range(new):
        m = n - new + 1 + j
        w = math.exp(-s)
        total = 1.0 + m * w
        common = 2.0 ** -15 + 2.0 ** -21 + 2 * n * 2.0 ** -24
        for dim, want, floor in ((0, 1.0, 2.0 ** -10), (1, m * w, m * (2.0 ** -10 * w + 1.5 * 2.0 ** -25))):
            want, bound = want / total, floor / total
            bound += want * (common + 2.0 ** -8 * 1.01)
            assert (np.abs(got[j, :, dim] - want) <= bound).all(), (j, dim, got[j, :, dim].tolist()[:2], want, bound)
        assert np.count_nonzero(got[j][:, 2:]) == 0
