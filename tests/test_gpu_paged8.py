"""The paged cache in 8 bits: append and read against the definition, bit for bit,
and attention against 64 bits.

Attention's tolerance, per output: half a bf16 step of the value (2^-8 |o|), plus

 - E * sum_i w_i |v_i|.  The weights enter the second product as a half (off by 2^-11)
   in three e5m2 parts of 3 significant bits: the first is cut (it leaves less than 2^-2
   of the weight's power of two), the second rounded (2^-6), the third rounded (2^-10):
   off by less than 2^-9; exp2's own error (2^-22); the sums of n terms in 32 bits
   (n * 2^-24 each, weights and values); and scores off by d, which move each weight and
   the sum by at most e^d - 1 < 2 d each: a dot product of hd products summed in fp32, for
   each of the two e4m3 parts of q (2 hd * 2^-24 * scale * sum |q||k|), roundings of the
   scaled score (2^-22 |s|: the query row's and the key's powers of two are exact, scale *
   log2 e, the product and the difference round), and what the two parts leave of q:
   nothing of an element within 2^-8 of the row's largest (8 significant bits are two
   e4m3's), else half of e4m3's smallest step, 2^-10, where the largest is at least 2^7:
   2^-17 of it.
   E = 2^-9 + 2^-21 + 4 d + 2 n 2^-24.
 - F * vmax, vmax the largest |v| of the sequence: a weight is kept relative to the
   largest that is known, times 2^3 at least, and its third part times 4 * 8 more; what
   is smaller than half of e5m2's smallest number, 2^-17, is lost, 2^-25 of the weight:
   n * 2^-25, times 2, since values are at most twice their row's largest after scaling
   by a power of two, and 2 for the sum that divides:
   F = n * 2^-23."""
import random

import numpy as np
import pytest

from gpu_common import torch_cuda
from test_gpu_paged import BATCHES, HEADER, HEADS, PAGE, Case, DevicePool, i32, pages_of

pytestmark = pytest.mark.gpu


def sv_():
    import speculative_decoding_verify_pass_gb300 as sv
    return sv


# --------------------------------------------------------- the definition ---
def e4m3(x):
    """Nearest e4m3 values (ties to even) of finite float64 x, |x| <= 464."""
    m, e = np.frexp(np.abs(x))
    step = np.exp2(np.maximum(e - 4.0, -9.0))
    return np.sign(x) * np.minimum(np.rint(np.abs(x) / step) * step, 448.0)


def quantised(x):
    """(codes' values, exponents) of rows [..][hd] (float64; NaN and infinities become NaN)."""
    x = np.asarray(x, dtype=np.float64)
    fine = np.isfinite(x)
    top = np.where(fine, np.abs(x), 0.0).max(-1)
    m, e = np.frexp(top)
    e = np.where(top > 0, e - 9 + (m > 0.875), -126)
    e = np.maximum(e, -126)
    return np.where(fine, e4m3(np.where(fine, x, 0.0) / np.exp2(e.astype(np.float64))[..., None]), np.nan), e


def dequantised(t):
    """What an 8-bit cache holds of bf16 rows, as a bf16 tensor (exact)."""
    torch = torch_cuda()
    c, e = quantised(t.double().numpy())
    return torch.from_numpy(c * np.exp2(e.astype(np.float64))[..., None]).bfloat16()


VALUES = np.array([(-1.0 if b & 128 else 1.0) * (np.nan if b & 127 == 127 else ((b & 7) * 2.0 ** -9 if b & 120 == 0 else (8 + (b & 7)) * 2.0 ** ((b >> 3 & 15) - 10)))
                   for b in range(256)])


def bits(codes):
    """e4m3 bytes of values."""
    table = {v: b for b, v in enumerate(VALUES) if b not in (127, 255) and not (v == 0 and b == 128)}
    return np.vectorize(lambda v: 127 if np.isnan(v) else table[v], otypes=[np.uint8])(codes)


def cache(pages, hkv, hd, seed=0):
    """A pool of random bytes: what the calls must leave alone."""
    torch = torch_cuda()
    g = torch.Generator(device="cuda").manual_seed(seed)
    new = lambda *s: torch.randint(0, 256, s, dtype=torch.uint8, device="cuda", generator=g)  # noqa: E731
    return new(pages, hkv, PAGE, hd).view(torch.float8_e4m3fn), new(pages, hkv, PAGE, hd).view(torch.float8_e4m3fn), new(pages, hkv, 2, PAGE)


# ----------------------------------------------------------- append, read ---
@pytest.mark.parametrize("rows,hkv,hd,count,fused", [(1, 1, 64, None, False), (3, 8, 128, 2, True), (77, 5, 64, 77, True),
                                                     (1000, 3, 128, 999, False), (3000, 2, 128, 9000, True), (6, 3, 64, 0, False),
                                                     (6, 3, 64, -4, False), (33, 1, 64, None, False)])
def test_append_writes_the_slots_and_nothing_else(rows, hkv, hd, count, fused):
    torch = torch_cuda()
    sv = sv_()
    torch.manual_seed(rows)
    pages = rows // PAGE + 5
    kp, vp, sc = cache(pages, hkv, hd, rows)
    if fused:
        qkv = torch.randn((rows, (2 + 2 * hkv) * hd + 8), device="cuda").bfloat16()
        k = qkv[:, 2 * hd:(2 + hkv) * hd].unflatten(1, (hkv, hd))
        v = qkv[:, (2 + hkv) * hd:(2 + 2 * hkv) * hd].unflatten(1, (hkv, hd))
    else:
        k, v = (torch.randn((rows, hkv, hd), device="cuda").bfloat16() for _ in range(2))
    v *= torch.exp2(torch.randint(-20, 20, (rows, hkv, 1), device="cuda").float()).bfloat16()
    slots = torch.randperm(pages * PAGE, device="cuda")[:rows].to(torch.int32)
    slots[::5] = -1 - slots[::5]                       # padding
    live = rows if count is None else max(0, min(rows, count))
    want = [t.view(torch.uint8).cpu().numpy().copy() for t in (kp, vp, sc)]
    at = slots.cpu().numpy()
    sel = np.nonzero((at >= 0) & (np.arange(rows) < live))[0]
    for pool, which, t in ((want[0], 0, k), (want[1], 1, v)):
        c, e = quantised(t[torch.from_numpy(sel).cuda()].double().cpu().numpy()) if len(sel) else (np.zeros((0, hkv, hd)), np.zeros((0, hkv)))
        for i, r in enumerate(sel):
            pool[at[r] // PAGE, :, at[r] % PAGE] = bits(c[i])
            want[2][at[r] // PAGE, :, which, at[r] % PAGE] = e[i] + 127
    err = i32([0])
    sv.spec_paged_append_fp8(k, v, slots, None if count is None else i32([count]), kp, vp, sc, err)
    for got, w in zip((kp, vp, sc), want):
        g = got.view(torch.uint8).cpu().numpy()
        # a zero may carry either sign's byte in the table's reading: compare as values
        same = (g == w) if got is sc else (g == w) | ((g & 127 == 0) & (w & 127 == 0))
        assert same.all()
    assert err.item() == 0


def test_append_of_edges():
    """Zeros, the smallest bf16 and nearly the largest, values on both sides of 448 * 2^e and of a
    tie, infinities and NaN."""
    torch = torch_cuda()
    sv = sv_()
    rows = [[0.0], [-0.0, 0.0], [2.0 ** -133], [2.0 ** -126, -2.0 ** -133], [3.0e38, 1.0], [448.0], [450.0], [-448.0, 1.0],
            [1.75, 1.7578125], [1.0, 17 / 16, 19 / 16, -17 / 16, 2.0 ** -10, 3 * 2.0 ** -10], [float("inf"), 2.0, -3.0], [float("nan"), 5.0, -float("inf")],
            [float("nan")] * 64, [448.0, 2.0 ** -10, 2.0 ** -9, 3 * 2.0 ** -10, 2.0 ** -6, 0.0151], [2.0 ** -118, 2.0 ** -133], [2.0 ** -117]]
    x = torch.zeros((len(rows), 1, 64), dtype=torch.bfloat16)
    for i, r in enumerate(rows):
        x[i, 0, :len(r)] = torch.tensor(r).bfloat16()
    kp, vp, sc = cache(1, 1, 64, 1)
    slots = torch.arange(len(rows), dtype=torch.int32, device="cuda")
    sv.spec_paged_append_fp8(x.cuda(), x.flip(2).cuda(), slots, None, kp, vp, sc)
    c, e = quantised(x.double().numpy())
    n = len(rows)
    assert (sc[0, 0, :, :n].cpu().numpy() == (e[:, 0] + 127)[None]).all()
    for pool, want in ((kp, c[:, 0]), (vp, c[:, 0, ::-1])):
        got = VALUES[pool[0, 0, :n].view(torch.uint8).cpu().numpy()]
        assert np.array_equal(got, want, equal_nan=True)
    # read back: the codes' values, and what the cache held is what it gives
    k, v = sv.spec_paged_read_fp8(slots, None, kp, vp, sc)
    want = c * np.exp2(e.astype(np.float64))[..., None]
    assert np.array_equal(k.double().cpu().numpy(), want, equal_nan=True)
    assert np.array_equal(v.double().cpu().numpy(), want[..., ::-1], equal_nan=True)
    # appending what was read changes nothing
    kp2, vp2, sc2 = cache(1, 1, 64, 1)
    sv.spec_paged_append_fp8(k, v, slots, None, kp2, vp2, sc2)
    k2, v2 = sv.spec_paged_read_fp8(slots, None, kp2, vp2, sc2)
    assert np.array_equal(k2.double().cpu().numpy(), want, equal_nan=True) and torch.equal(torch.nan_to_num(v2), torch.nan_to_num(v))
    # the largest bf16 rounds up to 256 * 2^120 = 2^128, which bf16 does not hold
    x = torch.full((1, 1, 64), torch.finfo(torch.bfloat16).max, dtype=torch.bfloat16, device="cuda")
    sv.spec_paged_append_fp8(x, -x, slots[:1], None, kp, vp, sc)
    assert (VALUES[kp[0, 0, 0].view(torch.uint8).cpu().numpy()] == 256).all() and (sc[0, 0, :, 0] == 247).all()
    k, v = sv.spec_paged_read_fp8(slots[:1], None, kp, vp, sc)
    assert torch.isposinf(k).all() and torch.isneginf(v).all()


@pytest.mark.parametrize("hkv,hd,rows", [(1, 64, 1), (3, 128, 70), (8, 64, 500), (5, 128, 2000)])
def test_read_of_any_bytes(hkv, hd, rows):
    """Every code under every scale: c * 2^(b - 127) rounded once to bf16."""
    torch = torch_cuda()
    sv = sv_()
    pages = 9
    kp, vp, sc = cache(pages, hkv, hd, 7)
    sc.view(-1)[:4 * 256] = torch.arange(4 * 256, device="cuda").remainder(256).to(torch.uint8) if sc.numel() >= 1024 else 0
    slots = torch.randint(0, pages * PAGE, (rows,), device="cuda").to(torch.int32)     # the same one twice too
    slots[3::7] = -1
    room = torch.full((rows, hkv + 1, hd), 3.0, dtype=torch.bfloat16, device="cuda")
    k, v = sv.spec_paged_read_fp8(slots, i32([rows - 1]), kp, vp, sc, d_k=room[:, :hkv])
    assert k.data_ptr() == room.data_ptr() and (room[:, hkv] == 3.0).all()
    at = slots.cpu().numpy()
    for got, pool, which in ((k, kp, 0), (v, vp, 1)):
        values = VALUES[pool.view(torch.uint8).cpu().numpy()]
        scale = np.exp2(sc[:, :, which].cpu().numpy().astype(np.float64) - 127)
        scale[sc[:, :, which].cpu().numpy() == 255] = np.nan
        g = got.cpu()
        for r in range(rows):
            if at[r] < 0 or r >= rows - 1:
                assert which == 1 or (g[r] == 3.0).all()
                continue
            p, t = at[r] // PAGE, at[r] % PAGE
            want = torch.from_numpy(values[p, :, t] * scale[p, :, t, None]).float().bfloat16()
            assert torch.equal(torch.nan_to_num(g[r], nan=77.0), torch.nan_to_num(want, nan=77.0)), r


def test_slots_outside_the_pool():
    torch = torch_cuda()
    sv = sv_()
    kp, vp, sc = cache(2, 1, 64)
    keep = [t.view(torch.uint8).clone() for t in (kp, vp, sc)]
    k = torch.ones((3, 1, 64), dtype=torch.bfloat16, device="cuda")
    err = i32([0])
    sv.spec_paged_append_fp8(k, k, i32([2 * PAGE, -1, 2 ** 31 - 1]), None, kp, vp, sc, err)
    assert err.item() == sv.SPEC_PAGED_BAD_PAGE
    assert all(torch.equal(t.view(torch.uint8), o) for t, o in zip((kp, vp, sc), keep))
    err, out = i32([0]), torch.full_like(k, 9.0)
    sv.spec_paged_read_fp8(i32([128, -5, 2 ** 31 - 1]), None, kp, vp, sc, d_k=out, d_v=out, d_error=err)
    assert err.item() == sv.SPEC_PAGED_BAD_PAGE and (out == 9.0).all()
    sv.spec_paged_append_fp8(k, k, i32([128, 6, 128]), None, kp, vp, sc)      # without an error word
    assert (sc[0, 0, :, 6] == 119).all()                                      # 1.0 = 256 * 2^-8


def test_a_rejected_draft_leaves_no_trace():
    """Positions appended beside others, cropped and appended again: the cache is that of the kept tokens alone."""
    torch = torch_cuda()
    sv = sv_()
    k, v = (torch.randn((100, 2, 64), device="cuda").bfloat16() for _ in range(2))
    slots = torch.arange(100, dtype=torch.int32, device="cuda")
    a, b = cache(2, 2, 64, 3), cache(2, 2, 64, 3)
    sv.spec_paged_append_fp8(k, v, slots, None, *a)
    sv.spec_paged_append_fp8(k[:60], v[:60], slots[:60], None, *b)
    sv.spec_paged_append_fp8(k[60:80] * 1000, v[60:80] * 1000, slots[60:80], None, *b)
    sv.spec_paged_append_fp8(k[60:], v[60:], slots[60:], None, *b)
    assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


# -------------------------------------------------------------- attention ---
class Case8(Case):
    """The bf16 tests' case, its keys and values in 8 bits: what the cache gives is what
    the reference uses.  Behind the lengths and in unused pages every byte is NaN."""

    def __init__(self, lens, new, hq, hkv, hd, spread=3, **kw):
        torch = torch_cuda()
        super().__init__(lens, new, hq, hkv, hd, **kw)
        g = torch.Generator().manual_seed(len(lens) + hd)
        d = self.d
        kp = torch.full(d["kp"].shape, 255, dtype=torch.uint8)
        vp = torch.full(d["vp"].shape, 255, dtype=torch.uint8)
        self.sc = torch.full((self.num_pages, hkv, 2, PAGE), 255, dtype=torch.uint8)
        self.kp8, self.vp8 = kp, vp
        for q, n in enumerate(lens):
            # tokens of different size
            self.v[q] = (self.v[q].float() * torch.exp2(torch.randint(-spread, spread + 1, (n, hkv, 1), generator=g).float())).bfloat16()
            self.place(q, torch.arange(n))
        self.upload()

    def place(self, q, t):
        """Positions t of sequence q, quantised, to the host's pools."""
        torch = torch_cuda()
        if not len(t):
            return
        page, o = self.tables_cpu[q, t // PAGE].long(), t % PAGE
        for pool, rows, which in ((self.kp8, self.k, 0), (self.vp8, self.v, 1)):
            c, e = quantised(rows[q][t].double().numpy())
            pool[page, :, o] = torch.from_numpy(c).float().to(torch.float8_e4m3fn).view(torch.uint8)
            self.sc[page, :, which, o] = torch.from_numpy(e + 127).to(torch.uint8)
            rows[q][t] = torch.from_numpy(c * np.exp2(e.astype(np.float64))[..., None]).bfloat16()

    def upload(self):
        torch = torch_cuda()
        self.d.update(kp=self.kp8.cuda().view(torch.float8_e4m3fn), vp=self.vp8.cuda().view(torch.float8_e4m3fn), sc=self.sc.cuda())

    def put(self, q, t, k=None, v=None):
        if k is not None:
            self.k[q][t] = k
        if v is not None:
            self.v[q][t] = v
        self.place(q, torch_cuda().tensor([t]))
        self.upload()

    def run(self, max_new=None, **kw):
        d = self.d
        return sv_().spec_paged_attention_fp8(d["q"], d["start"], d["len"], d["tables"], d["kp"], d["vp"], d["sc"],
                                              max_new or max(1, max(self.new)), **kw)

    def reference(self, scale=None):
        scale = self.hd ** -0.5 if scale is None else scale
        out = np.zeros((self.rows, self.hq, self.hd))
        bound = np.zeros_like(out)
        G = self.hq // self.hkv
        for q, (n, m) in enumerate(zip(self.lens, self.new)):
            k = self.k[q].double().numpy()
            v = self.v[q].double().numpy()
            vmax = np.where(np.isfinite(v), np.abs(v), 0.0).max((0, 2), initial=0.0)[:, None, None]
            for j in range(m):
                seen = n - m + j + 1
                r = self.start[q] + j
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
                d = (2 * self.hd * 2.0 ** -24 * a + z + 2.0 ** -22 * np.abs(s)).max(-1, keepdims=True)
                E = 2.0 ** -9 + 2.0 ** -21 + 4 * d + 2 * seen * 2.0 ** -24
                F = seen * 2.0 ** -23 * vmax
                out[r] = o.reshape(self.hq, self.hd)
                bound[r] = (2.0 ** -8 * np.abs(o) + (1 + 2.0 ** -8) * (E * ov + F)).reshape(self.hq, self.hd)
        return out, bound


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("batch", BATCHES, ids=lambda b: "-".join(map(str, b[0])))
def test_attention_matches_64_bits(heads, batch):
    c = Case8(batch[0], batch[1], *heads, seed=sum(batch[0]) + heads[0])
    c.check(c.run())


@pytest.mark.parametrize("lens,new,heads", [
    ([5000], [1], (32, 8, 128)), ([20011], [8], (8, 2, 128)), ([9000], [16], (8, 1, 64)), ([4104, 7], [8, 1], (32, 8, 128)),
    ([30000], [1], (2, 2, 64)), ([2500, 2600, 2700], [16, 1, 4], (64, 8, 128))])
def test_attention_of_long_caches(lens, new, heads):
    c = Case8(lens, new, *heads, seed=3)
    c.check(c.run())


def test_attention_of_1024_sequences():
    rng = random.Random(4)
    lens = [rng.choice([0, 1, 3, 64, 90, 200]) for _ in range(1024)]
    new = [rng.randint(0, min(n, 4)) for n in lens]
    c = Case8(lens, new, 8, 2, 64, seed=5)
    c.check(c.run())


def test_attention_rows_without_positions_are_zero():
    torch = torch_cuda()
    c = Case8([0, 2, 130], [3, 5, 2], 8, 2, 128, seed=6)
    got = c.run()
    c.check(got)
    assert torch.count_nonzero(got[:3 + 3]).item() == 0
    assert torch.count_nonzero(got[3 + 3:]).item() > 0


@pytest.mark.parametrize("hint", [1, 2, 16, 100000])
def test_max_new_is_a_hint(hint):
    c = Case8([300, 80, 513], [200, 1, 33], 8, 2, 64, seed=7)
    c.check(c.run(max_new=hint))
    c = Case8([400], [130], 12, 4, 128, seed=8)
    c.check(c.run(max_new=hint))


def test_attention_strides_scale_and_untouched_rows():
    torch = torch_cuda()
    c = Case8([90, 400], [3, 5], 16, 4, 128, seed=9, extra_rows=4)
    wide = torch.full((c.rows, (16 + 9) * 128), 3.0, dtype=torch.bfloat16, device="cuda")
    wide[:, :16 * 128] = c.d["q"].flatten(1)
    c.d["q"] = wide[:, :16 * 128].unflatten(1, (16, 128))
    room = torch.full((c.rows, 17, 128), -4.0, dtype=torch.bfloat16, device="cuda")
    out = room[:, :16]
    err = i32([0])
    got = c.run(scale=0.5, d_out=out, d_error=err)
    assert got is out and err.item() == 0
    c.check(out, scale=0.5)
    assert (room[:, 16] == -4.0).all() and (room[8:] == -4.0).all()
    assert (wide[:, 16 * 128:] == 3.0).all()


@pytest.mark.parametrize("heads", [(8, 2, 128), (4, 1, 64), (128, 1, 64), (64, 2, 128)])
@pytest.mark.parametrize("where", [0, 100, 200, 900, 1290])
@pytest.mark.parametrize("factor", [30.0, -30.0])
def test_attention_scores_that_jump(heads, where, factor):
    """Keys along (or against) one query so that its scores pass +-1000 late, early or in
    the block: the references have to follow."""
    hq, hkv, hd = heads
    c = Case8([1300], [4], hq, hkv, hd, seed=10, qscale=4.0)
    for t in range(where, min(1300, where + 3)):
        for h in range(hkv):
            x = c.q[1].view(hkv, hq // hkv, hd)[h, 1]
            k = c.k[0][t].clone()
            k[h] = (factor * x.float() / 4).bfloat16()
            c.k[0][t] = k
            c.place(0, torch_cuda().tensor([t]))
    c.upload()
    c.check(c.run())


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("g", [1, 16])
def test_attention_rising_scores(g, hd):
    """Every later key scores higher than all before it."""
    torch = torch_cuda()
    c = Case8([3000], [2], 4 * g, 1, hd, seed=11)
    x = c.q[0, 0].float()
    for t in range(0, 3000, 50):
        c.k[0][t] = (x * (t / 3000.0) * 20).bfloat16()[None]
    c.place(0, torch.arange(3000))
    c.upload()
    c.check(c.run())


@pytest.mark.parametrize("rise", [8, 24, 40])
@pytest.mark.parametrize("heads,new", [((8, 2, 128), 2), ((32, 2, 64), 8)])
def test_attention_values_that_grow(rise, heads, new):
    """Tokens whose values grow by powers of two along the sequence, in steps and at once:
    the scale that weights are kept at follows."""
    torch = torch_cuda()
    c = Case8([1500], [new], *heads, seed=13, spread=0)
    e = (torch.arange(1500) * rise // 1500).float()
    e[700] = rise
    c.v[0] = (c.v[0].float() * torch.exp2(e)[:, None, None]).bfloat16()
    c.place(0, torch.arange(1500))
    c.upload()
    c.check(c.run())
    c.v[0] = (c.v[0].float() * torch.exp2(-2 * e)[:, None, None]).bfloat16()      # and that shrink
    c.place(0, torch.arange(1500))
    c.upload()
    c.check(c.run())


def test_attention_behind_a_key_that_takes_most_of_the_weight():
    """A first key that takes most of the weight and whose value is 2^-9 of the others':
    what the rest adds, spread over 20000 keys of about equal weight, still shows."""
    torch = torch_cuda()
    c = Case8([20000], [1], 4, 1, 128, seed=14, spread=0, qscale=0.01)
    c.q[0] = c.q[0, 0]
    c.d["q"] = c.q.cuda()
    x = c.q[0, 0].float()
    c.k[0][0] = (x * 11.3 * 128 ** 0.5 / (x * x).sum()).bfloat16()[None]
    c.v[0][0] *= 2.0 ** -9
    c.v[0][1:] = (c.v[0][1:].float() + 0.5).bfloat16()
    c.place(0, torch.arange(20000))
    c.upload()
    out, bound = c.reference()
    assert np.abs(out).mean() > 4 * bound.mean()      # the bound can tell
    c.check(c.run())


@pytest.mark.parametrize("exponent", [60, -100])
def test_attention_large_and_small_values(exponent):
    torch = torch_cuda()
    c = Case8([700], [2], 8, 2, 128, seed=12)
    c.v[0] = (c.v[0].float() * 2.0 ** exponent).bfloat16()
    for h in range(2):
        c.k[0][300][h] = (0.5 * c.q[0].view(2, 4, 128)[h, 0].float()).bfloat16()
    c.place(0, torch.arange(700))
    c.upload()
    c.check(c.run())


@pytest.mark.parametrize("exponent", [50, -50])
def test_attention_queries_of_any_size(exponent):
    """A query row's power of two is its own: rows 2^100 apart, keys that bring the scores back."""
    torch = torch_cuda()
    c = Case8([500], [3], 8, 2, 64, seed=15)
    c.q[1] = (c.q[1].float() * 2.0 ** exponent).bfloat16()
    c.q[2, 3] = 0.0
    c.d["q"] = c.q.cuda()
    c.check(c.run(), rows=[0, 2])
    c.check(c.run(scale=2.0 ** (-exponent - 3)), rows=[1] if exponent > 0 else [], scale=2.0 ** (-exponent - 3))


@pytest.mark.parametrize("exponent", [90, -90])
@pytest.mark.parametrize("heads", [(8, 2, 64), (32, 2, 128)])
def test_attention_keys_of_any_size(exponent, heads):
    """Keys whose scales lie far from 1, queries that bring the scores back."""
    torch = torch_cuda()
    c = Case8([700, 130], [3, 2], *heads, seed=23)
    for q, n in enumerate(c.lens):
        c.k[q] = (c.k[q].float() * 2.0 ** exponent).bfloat16()
        c.place(q, torch.arange(n))
    c.q = (c.q.float() * 2.0 ** -exponent).bfloat16()
    c.d["q"] = c.q.cuda()
    c.upload()
    c.check(c.run())


@pytest.mark.parametrize("heads", [(8, 2, 64), (32, 2, 128), (65, 1, 128), (4, 4, 64)])
@pytest.mark.parametrize("seed", range(4))
def test_attention_nan_codes_and_scales_reach_the_rows_that_see_them(heads, seed):
    """NaN codes of either sign and scale bytes of 255 anywhere in the cache: a value's NaN in its
    dimension, a key's and a scale's in the whole row of every query head of its kv head."""
    c = Case8([300, 1, 129, 2100, 64], [8, 1, 3, 2, 1], *heads, seed=24 + seed)
    rng = random.Random(seed)
    for _ in range(6):
        q = rng.randrange(len(c.lens))
        n, h, d, nan = c.lens[q], rng.randrange(c.hkv), rng.randrange(c.hd), rng.choice([127, 255])
        t = n - 1 - rng.randint(0, min(n - 1, rng.choice([1, 9, n])))
        page, o = int(c.tables_cpu[q, t // PAGE]), t % PAGE
        kind = rng.choice(["value", "key", "values' scale", "keys' scale"])
        if kind == "value":
            c.vp8[page, h, o, d] = nan
            c.v[q][t, h, d] = float("nan")
        elif kind == "key":
            c.kp8[page, h, o, d] = nan
            c.k[q][t, h, d] = float("nan")
        else:
            c.sc[page, h, int(kind[0] == "v"), o] = 255
            c.k[q][t, h] = float("nan")
    c.upload()
    got = c.run().double().cpu().numpy()[:c.start[-1]]
    out, bound = (x[:c.start[-1]] for x in c.reference())
    seen = np.isnan(out)
    assert np.array_equal(np.isnan(got), seen) and (np.abs(got - out)[~seen] <= bound[~seen]).all()


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("n", [130, 136, 128, 300])
def test_attention_nonfinite_later_drafts_do_not_reach_earlier_rows(value, hd, n):
    """A drafted position's NaN key, value or scale is masked for the rows before it; rows
    that see the value are NaN in its dimensions."""
    torch = torch_cuda()
    c = Case8([n, 40], [6, 2], 8, 2, hd, seed=12)
    v = c.v[0][n - 3].clone()
    v[:, 5] = value
    c.put(0, n - 3, v=v)
    c.put(1, 39, v=torch.full_like(c.v[1][39], value))
    got = c.run()
    c.check(got, rows=[0, 1, 2, 6])
    for r in (3, 4, 5):
        assert torch.isnan(got[r, :, 5]).all()
        keep = [d for d in range(hd) if d != 5]
        assert torch.isfinite(got[r][:, keep]).all()
    assert torch.isnan(got[7]).all()
    c = Case8([n], [6], 8, 2, hd, seed=13)
    c.put(0, n - 3, k=torch.full((2, hd), value).bfloat16())
    got = c.run()
    c.check(got, rows=[0, 1, 2])
    assert torch.isnan(got[3:]).all()
    for which in (0, 1):
        c = Case8([n], [6], 8, 2, hd, seed=13)
        c.sc[int(c.tables_cpu[0, (n - 3) // PAGE]), :, which, (n - 3) % PAGE] = 255
        c.upload()
        got = c.run()
        c.check(got, rows=[0, 1, 2])
        assert torch.isnan(got[3:]).all()


def test_attention_of_a_nan_query_row_alone():
    torch = torch_cuda()
    for value in (float("nan"), float("inf")):
        c = Case8([200], [3], 8, 2, 128, seed=14)
        c.q[1, 2, 7] = value
        c.d["q"] = c.q.cuda()
        got = c.run()
        c.check(got, rows=[0, 2])
        assert torch.isnan(got[1, 2]).all() and torch.isfinite(got[1, [0, 1, 3, 4, 5, 6, 7]]).all()


def test_attention_bad_pages_lengths_and_rows():
    torch = torch_cuda()
    sv = sv_()
    base = Case8([200, 70, 300], [2, 1, 4], 8, 2, 128, seed=14)
    good = base.run()
    for page in (-1, base.num_pages, 2 ** 31 - 1, -2 ** 31):
        c = Case8([200, 70, 300], [2, 1, 4], 8, 2, 128, seed=14)
        c.d["tables"][1, 1] = page
        err = i32([0])
        got = c.run(d_error=err)
        assert err.item() == sv.SPEC_PAGED_BAD_PAGE
        c.check(got, rows=[0, 1, 3, 4, 5, 6])
        assert torch.isfinite(got).all()
        c.run()
    width = base.d["tables"].shape[1]
    for length in (-1, width * PAGE + 1, 2 ** 31 - 1, -2 ** 31):
        c = Case8([200, 70, 300], [2, 1, 4], 8, 2, 128, seed=14)
        c.d["len"][1] = length
        err, out = i32([0]), torch.full_like(good, 9.0)
        c.run(d_error=err, d_out=out)
        assert err.item() == sv.SPEC_PAGED_BAD_LENGTH
        assert (out[2] == 9.0).all()
        c.check(out, rows=[0, 1, 3, 4, 5, 6])
    for start, skipped, kept in (([0, 2, 3, 8], [3, 4, 5, 6], [0, 1, 2]), ([-1, 2, 3, 7], [0, 1], [2, 3, 4, 5, 6]),
                                 ([0, 2, 1, 7], [], [0]), ([0, 2, 3, -2 ** 31], [3, 4, 5, 6], [0, 1, 2])):
        c = Case8([200, 70, 300], [2, 1, 4], 8, 2, 128, seed=14)
        c.d["start"] = i32(start)
        err, out = i32([0]), torch.full_like(good, 9.0)
        c.run(d_error=err, d_out=out)
        assert err.item() == sv.SPEC_PAGED_BAD_ROWS
        assert all((out[r] == 9.0).all() for r in skipped)
        c.check(out, rows=kept)
    err = i32([77])
    c = Case8([200, 70, 300], [2, 1, 4], 8, 2, 128, seed=14)
    c.d["len"][1] = -1
    c.run(d_error=err)
    assert err.item() == 77                            # a word that holds a code keeps it


def test_attention_same_call_same_bits():
    torch = torch_cuda()
    c = Case8([5000, 300, 1], [4, 1, 1], 32, 8, 128, seed=15)
    a = c.run().view(torch.int16)
    for _ in range(5):
        assert torch.equal(a, c.run().view(torch.int16))


@pytest.mark.parametrize("heads,new", [((12, 2, 64), 8), ((32, 4, 128), 8), ((8, 2, 128), 8)])
def test_attention_of_ragged_blocks_in_many_calls(heads, new):
    """Short sequences whose blocks leave some of the softmax's warpgroups without rows, segment
    by segment: no wait gives up, and every call gives the same bits."""
    torch = torch_cuda()
    rng = random.Random(19)
    lens = [rng.randint(8, 400) for _ in range(120)]
    c = Case8(lens, [rng.randint(1, new) for _ in lens], *heads, seed=20)
    err, outs = i32([0]), [torch.empty_like(c.d["q"]) for _ in range(2)]
    first = c.run(max_new=new, d_error=err)
    c.check(first)
    for _ in range(40):
        for k in range(100):
            c.run(max_new=new, d_error=err, d_out=outs[k & 1])
        assert err.item() == 0
        live = c.start[-1]
        assert all(torch.equal(o[:live].view(torch.int16), first[:live].view(torch.int16)) for o in outs)


def test_refusals_of_the_binding():
    torch = torch_cuda()
    sv = sv_()
    c = Case8([2700], [4], 16, 2, 128, seed=16)
    need = sv.spec_paged_attention_fp8_workspace(16, 2, 128, 4, c.d["tables"].shape[1])
    work = torch.full((max(1, need),), 255, dtype=torch.uint8, device="cuda")    # NaN bits
    c.check(c.run(d_work=work))
    for bad in ([work[:need - 1]] if need else []) + [work.float()]:
        with pytest.raises(sv.SpecError):
            c.run(d_work=bad)
    for bad in (torch.empty((4, 16, 64), dtype=torch.bfloat16, device="cuda"), torch.empty((4, 16, 128), device="cuda"),
                torch.empty((16, 4, 128), dtype=torch.bfloat16, device="cuda").transpose(0, 1)):
        with pytest.raises(sv.SpecError):
            c.run(d_out=bad)
    d = dict(c.d)
    for over in (dict(kp=d["kp"].transpose(1, 2).contiguous().transpose(1, 2)), dict(vp=d["vp"][:1]), dict(kp=d["kp"].float().bfloat16()),
                 dict(sc=d["sc"].int()), dict(sc=d["sc"][:1]), dict(sc=d["sc"].transpose(2, 3).contiguous()), dict(q=d["q"].float()),
                 dict(len=d["len"].long()), dict(start=d["start"][:1]), dict(tables=d["tables"].t()), dict(sc=None)):
        c.d = dict(d, **over)
        with pytest.raises(sv.SpecError):
            c.run()
    c.d = d
    c.d["sc"] = d["sc"].view(torch.float8_e8m0fnu)
    c.d["kp"] = d["kp"].view(torch.uint8)
    c.check(c.run())
    k = torch.zeros((3, 2, 128), dtype=torch.bfloat16, device="cuda")
    s = i32([0, 1, 2])
    pools = (d["kp"], d["vp"], d["sc"])
    for bad in (lambda: sv.spec_paged_append_fp8(k, k[:2], s, None, *pools), lambda: sv.spec_paged_append_fp8(k, k, s[:2], None, *pools),
                lambda: sv.spec_paged_append_fp8(k.half(), k, s, None, *pools), lambda: sv.spec_paged_append_fp8(k, k, s, k, *pools),
                lambda: sv.spec_paged_append_fp8(k[:1].expand(3, 2, 128), k, s, None, *pools),
                lambda: sv.spec_paged_append_fp8(k, k, s, None, d["kp"], d["vp"][:2], d["sc"]),
                lambda: sv.spec_paged_read_fp8(s, None, *pools, d_k=k.half()), lambda: sv.spec_paged_read_fp8(s, None, *pools, d_v=k[:2]),
                lambda: sv.spec_paged_read_fp8(s.long(), None, *pools), lambda: sv.spec_paged_read_fp8(s.view(1, 3), None, *pools)):
        with pytest.raises(sv.SpecError):
            bad()


def test_attention_two_streams_at_once():
    torch = torch_cuda()
    a = Case8([6000, 50], [4, 1], 32, 8, 128, seed=17)
    b = Case8([900, 1200, 3], [2, 2, 2], 8, 2, 64, seed=18)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for _ in range(8):
        with torch.cuda.stream(s1):
            outs.append((a, a.run()))
        with torch.cuda.stream(s2):
            outs.append((b, b.run()))
    torch.cuda.synchronize()
    for c, got in outs[-4:]:
        c.check(got)
    for c, got in outs:
        last = [g for d, g in outs if d is c][-1]
        assert torch.equal(got.view(torch.int16), last.view(torch.int16))


def test_two_captured_graphs_replayed_together():
    torch = torch_cuda()
    cases = [Case8([5000, 200], [4, 2], 32, 8, 128, seed=21), Case8([3000, 900], [8, 1], 32, 8, 128, seed=22)]
    graphs, outs = [], []
    for c in cases:
        c.run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(c.run())
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(6):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for c, o in zip(cases, outs):
        c.check(o)


def test_pools_of_more_than_2_31_elements():
    """Pages whose codes lie past 32 bits: append, read and attention at the pool's end."""
    torch = torch_cuda()
    sv = sv_()
    pages = 540000                                     # x 64 x 64: 2.2e9 codes
    kp = torch.empty((pages, 1, PAGE, 64), dtype=torch.float8_e4m3fn, device="cuda")
    vp, sc = torch.empty_like(kp), torch.empty((pages, 1, 2, PAGE), dtype=torch.uint8, device="cuda")
    c = Case8([3000, 70], [3, 1], 4, 1, 64, seed=23)
    at = 0
    for q, n in enumerate(c.lens):
        for j in range(pages_of(n)):
            c.d["tables"][q, j] = c.tables_cpu[q, j] = pages - 1 - at
            at += 1
    slots = torch.cat([c.tables_cpu[q, torch.arange(n) // PAGE] * PAGE + torch.arange(n) % PAGE for q, n in enumerate(c.lens)])
    slots = slots.to(torch.int32).cuda()
    k, v = torch.cat(c.k).cuda(), torch.cat(c.v).cuda()
    c.d["kp"], c.d["vp"], c.d["sc"] = kp, vp, sc
    err = i32([0])
    sv.spec_paged_append_fp8(k, v, slots, None, kp, vp, sc, err)
    k2, v2 = sv.spec_paged_read_fp8(slots, None, kp, vp, sc, d_error=err)
    assert torch.equal(k, k2) and torch.equal(v, v2)   # what an 8-bit cache gave is kept exactly
    c.check(c.run(d_error=err))
    assert err.item() == 0
    del kp, vp, sc
    c.d.clear()
    torch.cuda.empty_cache()


def test_tables_at_the_border_of_whole_pairs():
    c = Case8([1024, 1000, 5, 0, 513], [4, 1, 2, 1, 16], 8, 2, 128, seed=24)
    out, bound = c.reference()
    for width in (16, 17, 18):
        c.d["tables"] = c.tables_cpu[:, :width].contiguous().cuda()
        g = c.run().float().cpu().numpy()
        assert np.all(np.abs(g[:c.start[-1]] - out[:c.start[-1]]) <= bound[:c.start[-1]])


# ---------------------------------------------------------- run together ----
class Cycle8:
    """A serving loop's state: step, turn, append, attend (two layers), over one cache in 8 bits."""

    def __init__(self, nseq, hq, hkv, hd, num_pages, width, cap, seed):
        torch = torch_cuda()
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.nseq, self.hq, self.hkv, self.hd, self.cap = nseq, hq, hkv, hd, cap
        self.dev = DevicePool(num_pages, nseq, width, 0, cap)
        self.pools = [cache(num_pages, hkv, hd, layer) for layer in range(2)]
        self.keep = torch.zeros(nseq, dtype=torch.int32, device="cuda")
        self.add = torch.zeros(nseq, dtype=torch.int32, device="cuda")
        self.qkv = torch.zeros((2, cap, hq + 2 * hkv, hd), dtype=torch.bfloat16, device="cuda")
        self.turned = torch.zeros((2, cap, hq + hkv, hd), dtype=torch.bfloat16, device="cuda")
        self.out = torch.full((2, cap, hq, hd), 5.0, dtype=torch.bfloat16, device="cuda")
        self.turns, self.gain = sv_().spec_rope_table(hd, 5e5, sv_().SPEC_ROPE_WAVELENGTH, 8.0)

    def run(self):
        sv, d, hq, hkv = sv_(), self.dev, self.hq, self.hkv
        d.step(self.keep, self.add)
        for layer in range(2):
            x, y = self.qkv[layer], self.turned[layer]
            sv.spec_rope(x[:, :hq + hkv], self.turns, d.start, d.len, gain=self.gain, d_out=y)
            sv.spec_paged_append_fp8(y[:, hq:], x[:, hq + hkv:], d.slots, d.start[-1:], *self.pools[layer], d.pool[1:])
            sv.spec_paged_attention_fp8(y[:, :hq], d.start, d.len, d.tables, *self.pools[layer], 8, d_out=self.out[layer],
                                        d_error=d.pool[1:])


def check_cycles(cyc, run, cycles, seed):
    torch = torch_cuda()
    sv = sv_()
    rng = random.Random(seed)
    n = cyc.nseq
    hist = [[[], []] for _ in range(n)]
    freq = cyc.turns.cpu().numpy().view(np.uint64).astype(np.float64) * 2.0 ** -64 * 2 * np.pi
    for cycle in range(cycles):
        keep, add = [], []
        for q in range(n):
            have = len(hist[q][0])
            keep.append(0 if rng.random() < 0.1 else max(0, have - rng.randint(0, 7)))
            add.append(rng.choice([0, 1, 4, 8]) if have else rng.choice([1, 20, 70]))
        cyc.keep.copy_(i32(keep))
        cyc.add.copy_(i32(add))
        cyc.qkv.copy_(torch.randn(cyc.qkv.shape, generator=cyc.g, device="cuda"))
        cyc.out.fill_(5.0)
        run()
        torch.cuda.synchronize()
        assert cyc.dev.pool[1].item() == 0
        start = [0]
        for a in add:
            start.append(start[-1] + a)
        assert cyc.dev.start.tolist() == start
        pos = [keep[q] + j for q in range(n) for j in range(add[q])]
        for layer in range(2):
            x, y = cyc.qkv[layer].cpu(), cyc.turned[layer].cpu()
            a = np.array(pos).reshape(-1, 1, 1) * freq
            u, w = (x[:start[-1], :cyc.hq + cyc.hkv].double().numpy()[..., s] for s in (slice(0, cyc.hd // 2), slice(cyc.hd // 2, None)))
            want = np.concatenate([u * np.cos(a) - w * np.sin(a), w * np.cos(a) + u * np.sin(a)], -1)
            size = np.concatenate([np.abs(u) + np.abs(w)] * 2, -1)
            got = y[:start[-1]].double().numpy()
            assert np.all(np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * size + 2.0 ** -134)
            c = Case8.__new__(Case8)
            c.hq, c.hkv, c.hd, c.start, c.rows = cyc.hq, cyc.hkv, cyc.hd, start, cyc.cap
            c.lens, c.new, c.k, c.v, c.q = [], add, [], [], y[:, :cyc.hq]
            for q in range(n):
                h = hist[q][layer]
                del h[keep[q]:]
                h += [(dequantised(y[r, cyc.hq:]), dequantised(x[r, cyc.hq + cyc.hkv:])) for r in range(start[q], start[q + 1])]
                c.lens.append(len(h))
                z = torch.zeros((0, cyc.hkv, cyc.hd), dtype=torch.bfloat16)
                c.k.append(torch.stack([a for a, _ in h]) if h else z)
                c.v.append(torch.stack([b for _, b in h]) if h else z)
                if h:                            # what the cache holds, read back
                    t = torch.arange(len(h), device="cuda")
                    slots = (cyc.dev.tables[q, t // PAGE] * PAGE + t % PAGE).to(torch.int32)
                    k, v = sv.spec_paged_read_fp8(slots, None, *cyc.pools[layer])
                    assert torch.equal(k.cpu(), c.k[-1]) and torch.equal(v.cpu(), c.v[-1])
            c.check(cyc.out[layer])
            assert (cyc.out[layer, start[-1]:] == 5.0).all()


def test_cycles_of_step_rope_append_attention():
    cyc = Cycle8(6, 8, 2, 64, 60, 10, 500, 1)
    check_cycles(cyc, cyc.run, 10, 2)


def test_cycles_replayed_from_a_graph():
    torch = torch_cuda()
    cyc = Cycle8(5, 12, 4, 128, 60, 12, 400, 3)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        cyc.run()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cyc.run()
    check_cycles(cyc, graph.replay, 8, 4)
