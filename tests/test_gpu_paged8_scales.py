"""Attention over the 8-bit cache where values differ in size by many powers of two:
what a row does not see, or gives next to no weight, changes nothing of what it does see.

The tolerance is test_gpu_paged8.py's, but for the part that is absolute.  A weight times
its value's scale 2^ev is kept relative to the largest such product C among the positions
that its row sees: the largest is kept at more than 2, or, for a row whose warpgroup has
others of up to 2^3 its size, at more than 2^-2.  As a half it is off by 2^-25 where halves
end, its third part by half of e5m2's smallest step over 128: (2^-25 + 2^-17 / 128) / 2^-2 C
= 1.5 * 2^-22 C for each of the n positions, times a code of at most 448.  F = n * 448 * 1.5 * 2^-22 * C.
And exp2 gives zero below 2^-126: n * 2^-126 times the largest value."""
import random

import numpy as np
import pytest

from gpu_common import torch_cuda
from test_gpu_paged8 import Case8, quantised

pytestmark = pytest.mark.gpu


class CaseSeen(Case8):
    """Bounds from what each row sees."""
    floor = 1.5 * 2.0 ** -22

    def reference(self, scale=None):
        scale = self.hd ** -0.5 if scale is None else scale
        out = np.zeros((self.rows, self.hq, self.hd))
        bound = np.zeros_like(out)
        G = self.hq // self.hkv
        for q, (n, m) in enumerate(zip(self.lens, self.new)):
            k, v = self.k[q].double().numpy(), self.v[q].double().numpy()
            ev = np.exp2(quantised(v)[1].astype(np.float64)).T[:, None, :]        # [kv head][1][position]
            for j in range(m):
                seen, r = n - m + j + 1, self.start[q] + j
                if seen <= 0:
                    continue
                x = self.q[r].double().numpy().reshape(self.hkv, G, self.hd)
                top = np.abs(x).max(-1, keepdims=True)
                left = np.where(np.abs(x) < 2.0 ** -8 * top, 2.0 ** -17 * top, 0.0)
                kk, vv = k[:seen], v[:seen]
                s = np.einsum("hgd,nhd->hgn", x, kk) * scale
                a = np.einsum("hgd,nhd->hgn", np.abs(x), np.abs(kk)) * scale
                z = np.einsum("hgd,nhd->hgn", left, np.abs(kk)) * scale
                w = np.exp(s - s.max(-1, keepdims=True))
                w /= w.sum(-1, keepdims=True)
                o = np.einsum("hgn,nhd->hgd", w, vv)
                ov = np.einsum("hgn,nhd->hgd", w, np.abs(vv))
                d = (2 * self.hd * 2.0 ** -24 * a + z + 2.0 ** -22 * np.abs(s))
                d = np.where(w > 0, d, 0.0).max(-1, keepdims=True)
                E = 2.0 ** -9 + 2.0 ** -21 + 4 * d + 2 * seen * 2.0 ** -24
                F = seen * 448 * self.floor * (w * ev[..., :seen]).max(-1, keepdims=True)
                F = F + seen * 2.0 ** -126 * np.abs(vv).max((0, 2))[:, None, None]
                out[r] = o.reshape(self.hq, self.hd)
                # half of bf16's least step where values end
                bound[r] = (2.0 ** -8 * np.abs(o) + (1 + 2.0 ** -8) * (E * ov + F) + 2.0 ** -134).reshape(self.hq, self.hd)
        return out, bound

    def tells(self, rows):
        """The bound is well below what it is compared with."""
        out, bound = self.reference()
        return all(np.abs(out[r]).mean() > 8 * bound[r].mean() for r in rows)

    def grow(self, q, t, exponent):
        """Values of positions t of sequence q times 2^exponent."""
        torch = torch_cuda()
        self.v[q][t] = (self.v[q][t].double() * torch.exp2(torch.as_tensor(exponent, dtype=torch.float64))).bfloat16()
        self.place(q, torch.as_tensor(t))


@pytest.mark.parametrize("exponent", [10, 17, 20, 24, 27, 30, 60, 100])
@pytest.mark.parametrize("heads,n,new", [((8, 2, 64), 130, 6), ((32, 8, 128), 300, 6), ((16, 2, 128), 2100, 8), ((64, 1, 64), 515, 4),
                                         ((128, 1, 128), 700, 2)])
def test_a_later_drafts_large_values_reach_only_the_rows_that_see_it(exponent, heads, n, new):
    """Finite values of any size at the last position: the rows before it are as without them."""
    c = CaseSeen([n, 40], [new, 2], *heads, seed=31)
    c.grow(0, [n - 1], exponent)
    c.grow(1, [39], exponent)
    c.upload()
    early = list(range(new - 1)) + [new]
    assert c.tells(early)
    c.check(c.run())
    c.check(c.run(), rows=early)


@pytest.mark.parametrize("exponent", [20, 27, 30, 60])
@pytest.mark.parametrize("where", [0, 100, 200, 900, 1290])
@pytest.mark.parametrize("heads", [(4, 4, 64), (8, 8, 128), (8, 1, 64)])
def test_a_large_value_that_gets_no_weight(exponent, where, heads):
    """A key against every query of its kv head (about e^-60 and less of their weight, far below
    2^-exponent), its value 2^exponent above the others': the others' weights keep their bits."""
    torch = torch_cuda()
    hq, hkv, hd = heads
    c = CaseSeen([1300], [4], hq, hkv, hd, seed=32, qscale=1.0)
    if hq > hkv:                                       # one direction that all of the head's queries share
        c.q[:4] = (c.q[:4].float() * 0.3 + c.q[0, 0].float()).bfloat16()
        c.d["q"] = c.q.cuda()
    k = c.k[0][where].clone()
    for h in range(hkv):
        y = c.q[:4].view(4, hkv, hq // hkv, hd)[:, h, 0].float()
        y = y.mean(0) if hq > hkv else y[0]
        k[h] = (-y * 70.0 * hd ** 0.5 / (y * y).sum()).bfloat16()
    c.k[0][where] = k
    c.grow(0, [where], exponent)
    c.upload()
    assert c.tells([0] if hq == hkv else range(4))
    c.check(c.run())


@pytest.mark.parametrize("rise", [8, 24, 40, 90])
@pytest.mark.parametrize("heads,new", [((8, 2, 128), 2), ((32, 2, 64), 8)])
def test_values_that_grow_and_shrink(rise, heads, new):
    """Along the sequence and at single positions, some of them drafts that early rows do not see."""
    torch = torch_cuda()
    e = (torch.arange(1500) * rise // 1500) - rise // 2
    e[700] = rise // 2
    e[1499] = rise
    for sign in (1, -1):
        c = CaseSeen([1500], [new], *heads, seed=33, spread=0)
        c.grow(0, torch.arange(1500), (sign * e)[:, None, None])
        c.upload()
        c.check(c.run())


@pytest.mark.parametrize("gap", [3, 40, 60, 100, 150])
@pytest.mark.parametrize("where", [0, 5, 140, 1290])
@pytest.mark.parametrize("value", [0.0, 2.0 ** -30, 2.0 ** -120])
def test_a_key_that_takes_nearly_all_weight_and_has_no_value(gap, where, value):
    """2^gap of the others' weight on a position of no value: what the others add is small and exact."""
    torch = torch_cuda()
    c = CaseSeen([1300], [2], 4, 2, 128, seed=34, qscale=0.05, spread=0)
    c.q[:2] = c.q[0, :1]                               # one direction for all rows
    c.d["q"] = c.q.cuda()
    x = c.q[0, 0].float()
    c.k[0][where] = (x * gap * 0.6931 * 128 ** 0.5 / (x * x).sum()).bfloat16()[None]
    c.v[0] = (c.v[0].float() + 0.5).bfloat16()
    c.v[0][where] = value
    c.place(0, torch.arange(1300))
    c.upload()
    # (fp32 has weights down to 2^-126)
    if gap < 120:
        assert value == 2.0 ** -30 or c.tells([0])
    c.check(c.run())


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("part", ["first", "last", "middle", "all", "odd"])
def test_values_of_zero(hd, part):
    """Positions without a value in the first chunks, the last, between, everywhere."""
    torch = torch_cuda()
    c = CaseSeen([1500, 100], [3, 1], 8, 2, hd, seed=35)
    at = dict(first=slice(0, 400), last=slice(900, 1500), middle=slice(300, 1200), all=slice(0, 1500), odd=slice(1, 1500, 2))[part]
    c.v[0][at] = 0.0
    c.place(0, torch.arange(1500))
    c.upload()
    got = c.run()
    c.check(got)
    if part == "all":
        assert torch.count_nonzero(got[:3]).item() == 0


@pytest.mark.parametrize("heads", [(8, 2, 64), (32, 8, 128), (65, 1, 128), (64, 2, 64)])
@pytest.mark.parametrize("seed", range(6))
def test_sizes_at_random(heads, seed):
    """Every position's values and keys of a size of their own, jumps of scores among them."""
    torch = torch_cuda()
    rng = random.Random(seed * 100 + heads[0])
    lens = [rng.randint(1, 1500) for _ in range(4)] + [rng.choice([2100, 5000])]
    new = [min(n, rng.randint(1, 9)) for n in lens]
    c = CaseSeen(lens, new, *heads, seed=36 + seed)
    g = torch.Generator().manual_seed(seed)
    for q, n in enumerate(lens):
        wide = rng.choice([5, 25, 60])
        c.v[q] = (c.v[q].float() * torch.exp2(torch.randint(-wide, wide + 1, (n, heads[1], 1), generator=g).float())).bfloat16()
        loud = torch.rand((n, heads[1], 1), generator=g) < 0.01
        c.k[q] = (c.k[q].float() * torch.where(loud, rng.choice([3.0, 20.0]), 1.0)).bfloat16()
        c.place(q, torch.arange(n))
    c.upload()
    c.check(c.run())


@pytest.mark.parametrize("exponent", [50, -50, -110])
def test_query_rows_of_different_size(exponent):
    """Every row's own power of two: row 1 is 2^exponent of the others, with scores as small or
    large as that makes them, and with a scale that brings them back."""
    torch = torch_cuda()
    c = CaseSeen([500], [3], 8, 2, 64, seed=15)
    c.q[1] = (c.q[1].float() * 2.0 ** exponent).bfloat16()
    c.q[2, 3] = 0.0
    c.d["q"] = c.q.cuda()
    c.check(c.run(), rows=[0, 1, 2] if exponent < 0 else [0, 2])
    scale = 2.0 ** (-exponent - 3)
    c.check(c.run(scale=scale), rows=[1], scale=scale)
