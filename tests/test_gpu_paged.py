"""The paged cache shared by many sequences: page tables and slots against a list
implementation, the append against indexing, attention against 64 bits.

Attention's tolerance, per output: half a bf16 step of the value (2^-8 |o|,
torch.finfo(bfloat16).eps / 2), plus E * sum_i w_i |v_i| for what happens in 32
bits: the softmax weights enter the second product as a bf16 high and low part
(off by at most 2^-16), exp2's own error (2^-22), scores off by d (a dot product
of hd exact products summed in fp32, hd * 2^-24 * scale * sum |q||k|, and two
roundings of the scaled score, 2^-23 |s|), which move each weight and the sum
by at most e^d - 1 < 2 d each, and the sums of n terms in 32 bits (n * 2^-24
each, weights and values).  E = 2^-16 + 2^-21 + 4 d + 2 n 2^-24."""
import random

import numpy as np
import pytest

from gpu_common import torch_cuda

pytestmark = pytest.mark.gpu

PAGE, HEADER = 64, 8


def sv_():
    import speculative_decoding_verify_pass_gb300 as sv
    return sv


def i32(x):
    torch = torch_cuda()
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def pages_of(n):
    return (n + PAGE - 1) // PAGE


# ------------------------------------------------------------ page tables ---
class ListPool:
    """The step's definition on Python lists."""

    def __init__(self, num_pages, nseq, width, fill):
        self.free = list(range(num_pages - 1, -1, -1))
        self.tables = [[fill] * width for _ in range(nseq)]
        self.len = [0] * nseq
        self.num_pages, self.width, self.error = num_pages, width, 0

    def step(self, keep, add, cap):
        n = len(self.len)
        code = 0
        if any(k < 0 or k > l or a < 0 or k + a > self.width * PAGE for k, a, l in zip(keep, add, self.len)):
            code = 1
        elif sum(add) > cap:
            code = 2
        else:
            have = len(self.free) + sum(max(0, pages_of(l) - pages_of(k + a)) for k, a, l in zip(keep, add, self.len))
            if sum(max(0, pages_of(k + a) - pages_of(l)) for k, a, l in zip(keep, add, self.len)) > have:
                code = 3
        if code:
            self.error = self.error or code
            return [0] * (n + 1), []
        for q in range(n):
            self.free += self.tables[q][pages_of(keep[q] + add[q]):pages_of(self.len[q])]
        start, slots = [0], []
        for q in range(n):
            for j in range(pages_of(self.len[q]), pages_of(keep[q] + add[q])):
                self.tables[q][j] = self.free.pop()
            for t in range(keep[q], keep[q] + add[q]):
                slots.append(self.tables[q][t // PAGE] * PAGE + t % PAGE)
            self.len[q] = keep[q] + add[q]
            start.append(len(slots))
        return start, slots


class DevicePool:
    def __init__(self, num_pages, nseq, width, fill, cap):
        torch = torch_cuda()
        self.pool = torch.full((HEADER + num_pages,), -5, dtype=torch.int32, device="cuda")
        self.tables = torch.full((nseq, width), fill, dtype=torch.int32, device="cuda")
        self.len = torch.zeros(nseq, dtype=torch.int32, device="cuda")
        self.start = torch.full((nseq + 1,), -7, dtype=torch.int32, device="cuda")
        self.slots = torch.full((cap,), -9, dtype=torch.int32, device="cuda")
        sv_().spec_pages_init(self.pool)

    def step(self, keep, add):
        sv_().spec_pages_step(self.pool, self.tables, self.len, keep, add, self.start, self.slots)


def same(ref, dev, start, slots):
    assert dev.start.tolist() == start
    got = dev.slots.tolist()
    assert got[:len(slots)] == slots
    pool = dev.pool.tolist()
    assert pool[0] == len(ref.free) and pool[1] == ref.error and pool[2:HEADER] == [0] * (HEADER - 2)
    assert pool[HEADER:HEADER + len(ref.free)] == ref.free
    assert dev.tables.tolist() == ref.tables
    assert dev.len.tolist() == ref.len


@pytest.mark.parametrize("nseq,width,num_pages,add_hi,cap", [
    (1, 3, 4, 70, 100), (2, 1, 2, 64, 128), (33, 9, 200, 300, 5000), (64, 20, 500, 16, 1024), (1000, 6, 3500, 100, 60000),
    (1024, 4, 4096, 256, 262144)])
def test_steps_match_the_definition(nseq, width, num_pages, add_hi, cap):
    """Random crops and growths, failures among them: everything equal after each step,
    slots behind the last row untouched."""
    rng = random.Random(nseq * 1000 + width)
    ref = ListPool(num_pages, nseq, width, -3)
    dev = DevicePool(num_pages, nseq, width, -3, cap)
    failed = 0
    for step in range(12):
        keep = [l if rng.random() < 0.5 else rng.randint(0, l) for l in ref.len]
        add = [0 if rng.random() < 0.3 else rng.randint(0, min(add_hi, width * PAGE - k)) for k in keep]
        if step == 5:
            keep[-1] = ref.len[-1] + 1          # a length out of range
        if step == 7:
            add[0] = width * PAGE - keep[0] + 1  # more pages than a table row holds
        if step == 8:
            add[0], keep[0] = -1, 0
        if step == 10:
            keep = [0] * nseq                    # every sequence retires
            add = [0] * nseq
        dev.slots.fill_(-9)
        start, slots = ref.step(keep, add, cap)
        dev.step(i32(keep), i32(add))
        same(ref, dev, start, slots)
        assert dev.slots.tolist()[len(slots):] == [-9] * (cap - len(slots))
        failed += start == [0] * (nseq + 1) and ref.error != 0
    assert failed >= 3


def test_step_shortage_and_too_many_rows_change_nothing():
    ref, dev = ListPool(6, 2, 8, 0), DevicePool(6, 2, 8, 0, 300)
    for keep, add in (([0, 0], [130, 100]), ([130, 100], [0, 29]), ([130, 129], [0, 100])):
        start, slots = ref.step(keep, add, 300)
        dev.step(i32(keep), i32(add))
        same(ref, dev, start, slots)
    assert ref.error == 3 and ref.len == [130, 129]
    dev.pool[1] = 0
    ref.error = 0
    start, slots = ref.step([0, 0], [301, 0], 300)
    dev.step(i32([0, 0]), i32([301, 0]))
    same(ref, dev, start, slots)
    assert ref.error == 2
    # pages that one sequence gives back serve the other in the same call; the first error stays
    start, slots = ref.step([0, 129], [0, 130], 300)
    dev.step(i32([0, 129]), i32([0, 130]))
    same(ref, dev, start, slots)
    assert ref.len == [0, 259] and dev.pool[1].item() == 2


def test_keep_may_be_the_lengths_themselves():
    ref, dev = ListPool(9, 3, 4, 0), DevicePool(9, 3, 4, 0, 200)
    for add in ([60, 64, 1], [5, 0, 63]):
        start, slots = ref.step(list(ref.len), add, 200)
        dev.step(dev.len, i32(add))
        same(ref, dev, start, slots)


def test_init_hands_out_page_zero_first():
    dev = DevicePool(300, 1, 4, 0, 200)
    assert dev.pool.tolist() == [300] + [0] * 7 + list(range(299, -1, -1))
    dev.step(i32([0]), i32([129]))
    assert dev.tables.tolist() == [[0, 1, 2, 0]]


@pytest.mark.parametrize("page", [-1, -2 ** 31, 9, 2 ** 25, 2 ** 26 + 3, 2 ** 31 - 1])
@pytest.mark.parametrize("nseq", [3, 1024])
def test_step_reports_pages_outside_the_pool(page, nseq):
    """A bad page that is held, taken or given back is reported, no slot on it lies in the
    pool (2^26 + 3 times 64 is 192 in 32 bits), and the append writes nothing through it."""
    sv = sv_()
    torch = torch_cuda()
    lens, rows = [60, 70, 64] + [0] * (nseq - 3), 30000 if nseq > 3 else 300

    def fresh():
        dev = DevicePool(9, nseq, 3, 0, rows)
        dev.step(i32([0] * nseq), i32(lens))
        assert dev.pool[1].item() == 0
        dev.slots.fill_(-9)
        return dev

    dev = fresh()                              # held: the entry that sequence 1's new rows fall on
    dev.tables[1, 1] = page
    dev.step(dev.len, i32([2, 3, 1] + [0] * (nseq - 3)))
    assert dev.pool[1].item() == sv.SPEC_PAGED_BAD_PAGE
    assert dev.start.tolist() == [0, 2, 5] + [6] * (nseq - 2)
    slots = dev.slots.tolist()
    assert slots[:2] == [60, 61] and slots[5] == 4 * 64 and slots[6:] == [-9] * (rows - 6)
    assert all(s >= 9 * 64 for s in slots[2:5])
    assert dev.len.tolist() == [62, 73, 65] + [0] * (nseq - 3)
    k = torch.ones((6, 1, 64), dtype=torch.bfloat16, device="cuda")
    kp = torch.zeros((9, 1, PAGE, 64), dtype=torch.bfloat16, device="cuda")
    vp, err = torch.zeros_like(kp), i32([0])
    sv.spec_paged_append(k, k, dev.slots[:6], dev.start[nseq:], kp, vp, err)
    assert err.item() == sv.SPEC_PAGED_BAD_PAGE
    assert kp.sum().item() == 3 * 64 and torch.equal(kp, vp)

    dev = fresh()                              # taken: the top of the stack
    dev.pool[HEADER + dev.pool[0].item() - 1] = page
    dev.step(dev.len, i32([0, 0, 2] + [0] * (nseq - 3)))
    assert dev.pool[1].item() == sv.SPEC_PAGED_BAD_PAGE
    assert all(s >= 9 * 64 for s in dev.slots.tolist()[:2])

    dev = fresh()                              # given back
    dev.tables[1, 1] = page
    dev.step(i32([60, 3, 64] + [0] * (nseq - 3)), i32([0] * nseq))
    assert dev.pool[1].item() == sv.SPEC_PAGED_BAD_PAGE and dev.pool[0].item() == 6


# ----------------------------------------------------------------- append ---
@pytest.mark.parametrize("rows,hkv,hd,count,fused", [(1, 1, 64, None, False), (3, 8, 128, 2, True), (77, 5, 64, 77, True),
                                                     (1000, 8, 128, 999, False), (5000, 2, 128, 9000, True), (6, 3, 64, 0, False),
                                                     (6, 3, 64, -4, False)])
def test_append_writes_the_slots_and_nothing_else(rows, hkv, hd, count, fused):
    torch = torch_cuda()
    sv = sv_()
    torch.manual_seed(rows)
    pages = rows // PAGE + 5
    kp = torch.randn((pages, hkv, PAGE, hd), device="cuda").bfloat16()
    vp = torch.randn((pages, hkv, PAGE, hd), device="cuda").bfloat16()
    if fused:
        qkv = torch.randn((rows, (2 + 2 * hkv) * hd + 8), device="cuda").bfloat16()
        k = qkv[:, 2 * hd:(2 + hkv) * hd].unflatten(1, (hkv, hd))
        v = qkv[:, (2 + hkv) * hd:(2 + 2 * hkv) * hd].unflatten(1, (hkv, hd))
    else:
        k, v = (torch.randn((rows, hkv, hd), device="cuda").bfloat16() for _ in range(2))
    k[0, 0, 0] = float("nan")
    slots = torch.randperm(pages * PAGE, device="cuda")[:rows].to(torch.int32)
    slots[::5] = -1 - slots[::5]                       # padding
    want_k, want_v = kp.clone(), vp.clone()
    live = rows if count is None else max(0, min(rows, count))
    for r in range(live):
        s = int(slots[r]) if rows < 100 else None
        if rows < 100 and s >= 0:
            want_k[s // PAGE, :, s % PAGE] = k[r]
            want_v[s // PAGE, :, s % PAGE] = v[r]
    if rows >= 100:
        sel = torch.nonzero((slots >= 0) & (torch.arange(rows, device="cuda") < live)).flatten()
        s = slots[sel].long()
        want_k[s // PAGE, :, s % PAGE] = k[sel]
        want_v[s // PAGE, :, s % PAGE] = v[sel]
    err = i32([0])
    sv.spec_paged_append(k, v, slots, None if count is None else i32([count]), kp, vp, err)
    assert torch.equal(kp.view(torch.int16), want_k.view(torch.int16))
    assert torch.equal(vp.view(torch.int16), want_v.view(torch.int16))
    assert err.item() == 0


def test_append_skips_slots_outside_the_pool():
    torch = torch_cuda()
    sv = sv_()
    kp = torch.zeros((2, 1, PAGE, 64), dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    k = torch.ones((3, 1, 64), dtype=torch.bfloat16, device="cuda")
    err = i32([0])
    sv.spec_paged_append(k, k, i32([2 * PAGE, 5, 2 ** 31 - 1]), None, kp, vp, err)
    assert err.item() == sv.SPEC_PAGED_BAD_PAGE
    assert kp.sum().item() == 64 and kp[0, 0, 5].sum().item() == 64 and torch.equal(kp, vp)
    sv.spec_paged_append(k, k, i32([128, 6, 128]), None, kp, vp)      # without an error word
    assert kp.sum().item() == 128


# -------------------------------------------------------------- attention ---
class Case:
    """Pools, tables and queries for the given lengths and new rows; pages
    shuffled, everything behind the lengths and every unused page NaN."""

    def __init__(self, lens, new, hq, hkv, hd, seed=0, garbage=float("nan"), extra_rows=0, qscale=2.0):
        torch = torch_cuda()
        g = torch.Generator().manual_seed(seed)
        self.lens, self.new, self.hq, self.hkv, self.hd = lens, new, hq, hkv, hd
        width = max(1, max(pages_of(n) for n in lens)) + 2
        self.num_pages = sum(pages_of(n) for n in lens) + 3
        perm = torch.randperm(self.num_pages, generator=g)
        self.k, self.v = [], []
        kp = torch.full((self.num_pages, hkv, PAGE, hd), garbage).bfloat16()
        vp = torch.full((self.num_pages, hkv, PAGE, hd), garbage).bfloat16()
        tables = torch.full((len(lens), width), 2 ** 31 - 1, dtype=torch.int32)
        at = 0
        for q, n in enumerate(lens):
            k = torch.randn((n, hkv, hd), generator=g).bfloat16()
            v = torch.randn((n, hkv, hd), generator=g).bfloat16()
            self.k.append(k)
            self.v.append(v)
            for j in range(pages_of(n)):
                page = int(perm[at])
                at += 1
                tables[q, j] = page
                part = slice(j * PAGE, min(n, (j + 1) * PAGE))
                kp[page, :, :part.stop - part.start] = k[part].transpose(0, 1)
                vp[page, :, :part.stop - part.start] = v[part].transpose(0, 1)
        self.start = [0]
        for m in new:
            self.start.append(self.start[-1] + m)
        self.rows = self.start[-1] + extra_rows
        self.q = (qscale * torch.randn((self.rows, hq, hd), generator=g)).bfloat16()
        self.tables_cpu = tables
        self.d = dict(q=self.q.cuda(), start=i32(self.start), len=i32(lens), tables=tables.cuda(), kp=kp.cuda(), vp=vp.cuda())

    def put(self, q, t, k=None, v=None):
        """Set position t of sequence q's keys or values (all heads)."""
        page, o = int(self.tables_cpu[q, t // PAGE]), t % PAGE
        if k is not None:
            self.k[q][t] = k
            self.d["kp"][page, :, o] = k
        if v is not None:
            self.v[q][t] = v
            self.d["vp"][page, :, o] = v

    def run(self, max_new=None, **kw):
        d = self.d
        return sv_().spec_paged_attention(d["q"], d["start"], d["len"], d["tables"], d["kp"], d["vp"],
                                          max_new or max(1, max(self.new)), **kw)

    def reference(self, scale=None):
        """(out, bound) in 64 bits, rows of sequences only."""
        scale = self.hd ** -0.5 if scale is None else scale
        out = np.zeros((self.rows, self.hq, self.hd))
        bound = np.zeros_like(out)
        G = self.hq // self.hkv
        for q, (n, m) in enumerate(zip(self.lens, self.new)):
            k = self.k[q].double().numpy()
            v = self.v[q].double().numpy()
            for j in range(m):
                seen = n - m + j + 1
                r = self.start[q] + j
                if seen <= 0:
                    continue
                x = self.q[r].double().numpy().reshape(self.hkv, G, self.hd)
                kk, vv = k[:seen], v[:seen]
                s = np.einsum("hgd,nhd->hgn", x, kk) * scale
                a = np.einsum("hgd,nhd->hgn", np.abs(x), np.abs(kk)) * scale
                w = np.exp(s - s.max(-1, keepdims=True))
                w /= w.sum(-1, keepdims=True)
                o = np.einsum("hgn,nhd->hgd", w, vv)
                ov = np.einsum("hgn,nhd->hgd", w, np.abs(vv))
                d = (self.hd * 2.0 ** -24 * a + 2.0 ** -23 * np.abs(s)).max(-1, keepdims=True)
                E = 2.0 ** -16 + 2.0 ** -21 + 4 * d + 2 * seen * 2.0 ** -24
                out[r] = o.reshape(self.hq, self.hd)
                bound[r] = (2.0 ** -8 * np.abs(o) + E * (1 + 2.0 ** -8) * ov).reshape(self.hq, self.hd)
        return out, bound

    def check(self, got, scale=None, rows=None):
        out, bound = self.reference(scale)
        g = got.float().cpu().numpy().astype(np.float64)
        rows = range(self.start[-1]) if rows is None else rows
        for r in rows:
            err = np.abs(g[r] - out[r])
            assert np.all(err <= bound[r]), (r, float((err - bound[r]).max()), float(err.max()))


HEADS = [(4, 4, 64), (32, 8, 128), (8, 1, 128), (16, 16, 128), (7, 1, 64), (18, 3, 128), (20, 4, 64), (64, 1, 128), (128, 1, 64),
         (40, 8, 64)]
BATCHES = [([1], [1]), ([64], [1]), ([65], [2]), ([128], [8]), ([129], [16]), ([127], [5]), ([192], [16]),
           ([1, 700, 64, 0, 128, 1300, 129], [1, 8, 3, 0, 16, 1, 2]), ([300, 0, 40], [0, 0, 1]), ([15, 16, 17, 33], [15, 16, 16, 3])]


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("batch", BATCHES, ids=lambda b: "-".join(map(str, b[0])))
def test_attention_matches_64_bits(heads, batch):
    c = Case(batch[0], batch[1], *heads, seed=sum(batch[0]) + heads[0])
    c.check(c.run())


@pytest.mark.parametrize("lens,new,heads", [
    ([5000], [1], (32, 8, 128)), ([20011], [8], (8, 2, 128)), ([9000], [16], (8, 1, 64)), ([4104, 7], [8, 1], (32, 8, 128)),
    ([30000], [1], (2, 2, 64)), ([2500, 2600, 2700], [16, 1, 4], (64, 8, 128))])
def test_attention_of_long_caches(lens, new, heads):
    c = Case(lens, new, *heads, seed=3)
    c.check(c.run())


def test_attention_of_1024_sequences():
    rng = random.Random(4)
    lens = [rng.choice([0, 1, 3, 64, 90, 200]) for _ in range(1024)]
    new = [rng.randint(0, min(n, 4)) for n in lens]
    c = Case(lens, new, 8, 2, 64, seed=5)
    c.check(c.run())


def test_attention_rows_without_positions_are_zero():
    torch = torch_cuda()
    c = Case([0, 2, 130], [3, 5, 2], 8, 2, 128, seed=6)
    got = c.run()
    c.check(got)
    assert torch.count_nonzero(got[:3 + 3]).item() == 0
    assert torch.count_nonzero(got[3 + 3:]).item() > 0


@pytest.mark.parametrize("hint", [1, 2, 16, 100000])
def test_max_new_is_a_hint(hint):
    """Blocks longer than max_new, and longer than 16: the same answer."""
    c = Case([300, 80, 513], [200, 1, 33], 8, 2, 64, seed=7)
    c.check(c.run(max_new=hint))
    c = Case([400], [130], 12, 4, 128, seed=8)
    c.check(c.run(max_new=hint))


def test_attention_strides_scale_and_untouched_rows():
    torch = torch_cuda()
    c = Case([90, 400], [3, 5], 16, 4, 128, seed=9, extra_rows=4)
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


@pytest.mark.parametrize("where", [0, 100, 200, 900, 1290])
@pytest.mark.parametrize("factor", [30.0, -30.0])
def test_attention_scores_that_jump(where, factor):
    """Keys along (or against) the query so that scores pass +-1000 late, early
    or in the block: the running maximum has to follow."""
    c = Case([1300], [4], 8, 2, 128, seed=10, qscale=4.0)
    for t in range(where, min(1300, where + 3)):
        for h in range(2):
            x = c.q[1].view(2, 4, 128)[h, 1]
            k = c.k[0][t].clone()
            k[h] = (factor * x.float() / 4).bfloat16()
            c.put(0, t, k=k)
    c.check(c.run())


def test_attention_rising_scores():
    """Every later key scores higher than all before it."""
    torch = torch_cuda()
    c = Case([3000], [2], 4, 1, 64, seed=11)
    x = c.q[0, 0].float()
    for t in range(0, 3000, 50):
        c.put(0, t, k=(x * (t / 3000.0) * 20).bfloat16()[None])
    c.check(c.run())


@pytest.mark.parametrize("exponent", [60, -100])
def test_attention_large_and_small_values(exponent):
    """Values of 2^60 under a weight of about 2^32 times the first key's, and of 2^-100."""
    c = Case([700], [2], 8, 2, 128, seed=12)
    c.v[0] *= 2.0 ** exponent
    c.d["vp"] *= 2.0 ** exponent
    for h in range(2):
        k = c.k[0][300].clone()
        k[h] = (0.5 * c.q[0].view(2, 4, 128)[h, 0].float()).bfloat16()
        c.put(0, 300, k=k)
    c.check(c.run())


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("n", [130, 136, 128, 300])
def test_attention_nonfinite_later_drafts_do_not_reach_earlier_rows(value, hd, n):
    """A drafted position's non-finite key or value is masked for the rows before
    it; rows that see the value are non-finite in its dimensions."""
    torch = torch_cuda()
    c = Case([n, 40], [6, 2], 8, 2, hd, seed=12)
    v = c.v[0][n - 3].clone()
    v[:, 5] = value
    c.put(0, n - 3, v=v)
    v2 = c.v[1][39].clone()
    v2[:] = value
    c.put(1, 39, v=v2)
    got = c.run()
    c.check(got, rows=[0, 1, 2, 6])
    for r in (3, 4, 5):
        assert not torch.isfinite(got[r, :, 5]).any()
        keep = [d for d in range(hd) if d != 5]
        assert torch.isfinite(got[r][:, keep]).all()
    assert not torch.isfinite(got[7]).any()
    c = Case([n], [6], 8, 2, hd, seed=13)
    c.put(0, n - 3, k=torch.full((2, hd), value).bfloat16())
    c.check(c.run(), rows=[0, 1, 2])


def test_attention_bad_pages_lengths_and_rows():
    torch = torch_cuda()
    sv = sv_()
    base = Case([200, 70, 300], [2, 1, 4], 8, 2, 128, seed=14)
    good = base.run()
    for page in (-1, base.num_pages, 2 ** 31 - 1, -2 ** 31):
        c = Case([200, 70, 300], [2, 1, 4], 8, 2, 128, seed=14)
        c.d["tables"][1, 1] = page
        err = i32([0])
        got = c.run(d_error=err)
        assert err.item() == sv.SPEC_PAGED_BAD_PAGE
        c.check(got, rows=[0, 1, 3, 4, 5, 6])
        assert torch.isfinite(got).all()
        c.run()
    width = base.d["tables"].shape[1]
    for length in (-1, width * PAGE + 1, 2 ** 31 - 1, -2 ** 31):
        c = Case([200, 70, 300], [2, 1, 4], 8, 2, 128, seed=14)
        c.d["len"][1] = length
        err, out = i32([0]), torch.full_like(good, 9.0)
        c.run(d_error=err, d_out=out)
        assert err.item() == sv.SPEC_PAGED_BAD_LENGTH
        assert (out[2] == 9.0).all()
        c.check(out, rows=[0, 1, 3, 4, 5, 6])
    for start, skipped, kept in (([0, 2, 3, 8], [3, 4, 5, 6], [0, 1, 2]), ([-1, 2, 3, 7], [0, 1], [2, 3, 4, 5, 6]),
                                 ([0, 2, 1, 7], [], [0]), ([0, 2, 3, -2 ** 31], [3, 4, 5, 6], [0, 1, 2])):
        c = Case([200, 70, 300], [2, 1, 4], 8, 2, 128, seed=14)
        c.d["start"] = i32(start)
        err, out = i32([0]), torch.full_like(good, 9.0)
        c.run(d_error=err, d_out=out)
        assert err.item() == sv.SPEC_PAGED_BAD_ROWS
        assert all((out[r] == 9.0).all() for r in skipped)
        c.check(out, rows=kept)
    err = i32([77])
    c = Case([200, 70, 300], [2, 1, 4], 8, 2, 128, seed=14)
    c.d["len"][1] = -1
    c.run(d_error=err)
    assert err.item() == 77                            # a word that holds a code keeps it


def test_attention_same_call_same_bits():
    torch = torch_cuda()
    c = Case([5000, 300, 1], [4, 1, 1], 32, 8, 128, seed=15)
    a = c.run().view(torch.int16)
    for _ in range(5):
        assert torch.equal(a, c.run().view(torch.int16))


def test_attention_workspace_from_the_caller_and_its_refusals():
    torch = torch_cuda()
    sv = sv_()
    c = Case([2700], [4], 16, 2, 128, seed=16)
    need = sv.spec_paged_attention_workspace(16, 2, 128, 4, c.d["tables"].shape[1])
    assert need > 0
    work = torch.full((need,), 255, dtype=torch.uint8, device="cuda")    # NaN bits
    c.check(c.run(d_work=work))
    for bad in (work[:need - 1], work.float()):
        with pytest.raises(sv.SpecError):
            c.run(d_work=bad)
    with pytest.raises(sv.SpecError):
        c.run(d_out=torch.empty((4, 16, 64), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(sv.SpecError):
        c.run(d_out=torch.empty((4, 16, 128), dtype=torch.float32, device="cuda"))
    with pytest.raises(sv.SpecError):
        c.run(d_out=torch.empty((16, 4, 128), dtype=torch.bfloat16, device="cuda").transpose(0, 1))
    for name in ("kp", "vp"):
        keep = c.d[name]
        c.d[name] = keep.transpose(1, 2).contiguous().transpose(1, 2)
        with pytest.raises(sv.SpecError):
            c.run()
        c.d[name] = keep


def test_attention_two_streams_at_once():
    torch = torch_cuda()
    a = Case([6000, 50], [4, 1], 32, 8, 128, seed=17)
    b = Case([900, 1200, 3], [2, 2, 2], 8, 2, 64, seed=18)
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


def test_pools_of_more_than_2_31_elements():
    """Pages whose elements lie past 32 bits: append and attention at the pool's end."""
    torch = torch_cuda()
    sv = sv_()
    pages = 540000                                     # x 64 x 64: 2.2e9 elements
    kp = torch.empty((pages, 1, PAGE, 64), dtype=torch.bfloat16, device="cuda")
    vp = torch.empty_like(kp)
    c = Case([3000, 70], [3, 1], 4, 1, 64, seed=23)
    at = 0
    for q, n in enumerate(c.lens):
        for j in range(pages_of(n)):
            c.d["tables"][q, j] = c.tables_cpu[q, j] = pages - 1 - at
            at += 1
    slots = torch.cat([c.tables_cpu[q, torch.arange(n) // PAGE] * PAGE + torch.arange(n) % PAGE for q, n in enumerate(c.lens)])
    k, v = torch.cat(c.k).cuda(), torch.cat(c.v).cuda()
    c.d["kp"], c.d["vp"] = kp, vp
    err = i32([0])
    sv.spec_paged_append(k, v, slots.to(torch.int32).cuda(), None, kp, vp, err)
    c.check(c.run(d_error=err))
    assert err.item() == 0
    del kp, vp
    c.d.clear()
    torch.cuda.empty_cache()


def test_tables_at_the_border_of_whole_pairs():
    """Tables of 16 pages keep a pair on one CTA, of 17 split it: the same answer to the tolerance."""
    torch = torch_cuda()
    sv = sv_()
    c = Case([1024, 1000, 5, 0, 513], [4, 1, 2, 1, 16], 8, 2, 128, seed=24)
    out, bound = c.reference()
    for width in (16, 17, 18):
        c.d["tables"] = c.tables_cpu[:, :width].contiguous().cuda()
        assert (sv.spec_paged_attention_workspace(8, 2, 128, 16, width) == 0) == (width <= 16)
        g = c.run().float().cpu().numpy()
        assert np.all(np.abs(g[:c.start[-1]] - out[:c.start[-1]]) <= bound[:c.start[-1]])


# ---------------------------------------------------------- run together ----
class Cycle:
    """A serving loop's state: step, append to two layers, attend both."""

    def __init__(self, nseq, hq, hkv, hd, num_pages, width, cap, seed):
        torch = torch_cuda()
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.nseq, self.hq, self.hkv, self.hd, self.cap = nseq, hq, hkv, hd, cap
        self.dev = DevicePool(num_pages, nseq, width, 0, cap)
        self.pools = [[torch.full((num_pages, hkv, PAGE, hd), float("nan"), dtype=torch.bfloat16, device="cuda")
                       for _ in range(2)] for _ in range(2)]
        self.keep = torch.zeros(nseq, dtype=torch.int32, device="cuda")
        self.add = torch.zeros(nseq, dtype=torch.int32, device="cuda")
        self.qkv = torch.zeros((2, cap, (hq + 2 * hkv) * hd), dtype=torch.bfloat16, device="cuda")
        self.out = torch.full((2, cap, hq, hd), 5.0, dtype=torch.bfloat16, device="cuda")

    def new_rows(self):
        torch = torch_cuda()
        self.qkv.copy_(torch.randn(self.qkv.shape, generator=self.g, device="cuda"))

    def run(self):
        sv, d = sv_(), self.dev
        d.step(self.keep, self.add)
        for layer in range(2):
            hq, hkv, hd = self.hq, self.hkv, self.hd
            x = self.qkv[layer].unflatten(1, (hq + 2 * hkv, hd))
            kp, vp = self.pools[layer]
            sv.spec_paged_append(x[:, hq:hq + hkv], x[:, hq + hkv:], d.slots, d.start[-1:], kp, vp, d.pool[1:])
            sv.spec_paged_attention(x[:, :hq], d.start, d.len, d.tables, kp, vp, 8, d_out=self.out[layer],
                                    d_error=d.pool[1:])


def check_cycles(cyc, run, cycles, seed):
    """Runs random accept/reject cycles, keeping each sequence's true keys and values on the host."""
    torch = torch_cuda()
    rng = random.Random(seed)
    n = cyc.nseq
    hist = [[[], []] for _ in range(n)]              # per sequence and layer: list of (k, v)
    for cycle in range(cycles):
        keep, add = [], []
        for q in range(n):
            have = len(hist[q][0])
            k = 0 if rng.random() < 0.1 else max(0, have - rng.randint(0, 7))
            keep.append(k)
            add.append(rng.choice([0, 1, 4, 8]) if have else rng.choice([1, 20, 70]))
        cyc.keep.copy_(i32(keep))
        cyc.add.copy_(i32(add))
        cyc.new_rows()
        cyc.out.fill_(5.0)
        run()
        torch.cuda.synchronize()
        assert cyc.dev.pool[1].item() == 0
        start = [0]
        for a in add:
            start.append(start[-1] + a)
        assert cyc.dev.start.tolist() == start
        for layer in range(2):
            x = cyc.qkv[layer].unflatten(1, (cyc.hq + 2 * cyc.hkv, cyc.hd)).cpu()
            c = Case.__new__(Case)
            c.hq, c.hkv, c.hd, c.start, c.rows = cyc.hq, cyc.hkv, cyc.hd, start, cyc.cap
            c.lens, c.new, c.k, c.v, c.q = [], add, [], [], x[:, :cyc.hq]
            for q in range(n):
                h = hist[q][layer]
                del h[keep[q]:]
                h += [(x[r, cyc.hq:cyc.hq + cyc.hkv], x[r, cyc.hq + cyc.hkv:]) for r in range(start[q], start[q + 1])]
                c.lens.append(len(h))
                z = torch.zeros((0, cyc.hkv, cyc.hd), dtype=torch.bfloat16)
                c.k.append(torch.stack([a for a, _ in h]) if h else z)
                c.v.append(torch.stack([b for _, b in h]) if h else z)
            c.check(cyc.out[layer])
            assert (cyc.out[layer, start[-1]:] == 5.0).all()


def test_cycles_of_step_append_attention():
    cyc = Cycle(6, 8, 2, 64, 60, 10, 500, 1)
    check_cycles(cyc, cyc.run, 10, 2)


def test_cycles_replayed_from_a_graph():
    """One captured cycle, replayed with other lengths, accepts and rows."""
    torch = torch_cuda()
    cyc = Cycle(5, 12, 4, 128, 60, 12, 400, 3)
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


def test_two_captured_graphs_replayed_together():
    """Two graphs whose calls took their scratch from torch's allocator, replayed on two streams at once."""
    torch = torch_cuda()
    cases = [Case([5000, 200], [4, 2], 32, 8, 128, seed=21), Case([3000, 900], [8, 1], 32, 8, 128, seed=22)]
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


def test_paged_attention_agrees_with_the_verify_pass_layout():
    """The handle's own cache rows, moved into pages, give the pages' layout:
    what spec_kv_export returns appends as it is."""
    torch = torch_cuda()
    import synth
    from conftest import small_gqa_cfg
    from gpu_common import make_model
    sv = sv_()
    cfg = small_gqa_cfg()
    m = make_model(cfg, synth.make_weights(cfg))
    m.prefill(synth.prompt(cfg, 100))
    k, v = m.kv_export(sv.SPEC_CACHE_TARGET, 1, 100)
    m.close()
    k = torch.from_numpy(k.view(np.int16).copy()).cuda().view(torch.bfloat16)
    v = torch.from_numpy(v.view(np.int16).copy()).cuda().view(torch.bfloat16)
    dev = DevicePool(4, 1, 3, 0, 100)
    dev.step(i32([0]), i32([100]))
    kp = torch.zeros((4, cfg.n_kv_heads, PAGE, cfg.head_dim), dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    sv.spec_paged_append(k, v, dev.slots, None, kp, vp)
    q = torch.randn((5, cfg.n_heads, cfg.head_dim), device="cuda").bfloat16()
    got = sv.spec_paged_attention(q, i32([0, 5]), dev.len, dev.tables, kp, vp, 5)
    c = Case.__new__(Case)
    c.hq, c.hkv, c.hd, c.start, c.rows, c.lens, c.new = cfg.n_heads, cfg.n_kv_heads, cfg.head_dim, [0, 5], 5, [100], [5]
    c.k, c.v, c.q = [k.cpu()], [v.cpu()], q.cpu()
    c.check(got)


def test_binding_refuses_what_the_kernels_cannot_read():
    torch = torch_cuda()
    sv = sv_()
    c = Case([100], [2], 8, 2, 64, seed=19)
    d = c.d
    with pytest.raises(sv.SpecError):
        sv.spec_paged_attention(d["q"].float(), d["start"], d["len"], d["tables"], d["kp"], d["vp"], 2)
    with pytest.raises(sv.SpecError):
        sv.spec_paged_attention(d["q"], d["start"].long(), d["len"], d["tables"], d["kp"], d["vp"], 2)
    with pytest.raises(sv.SpecError):
        sv.spec_paged_attention(d["q"], d["start"][:1], d["len"], d["tables"], d["kp"], d["vp"], 2)
    with pytest.raises(sv.SpecError):
        sv.spec_paged_attention(d["q"], d["start"], d["len"], d["tables"], d["kp"], d["vp"][:1], 2)
    with pytest.raises(sv.SpecError):
        sv.spec_paged_attention(d["q"].transpose(1, 2).contiguous().transpose(1, 2), d["start"], d["len"], d["tables"],
                                d["kp"], d["vp"], 2)
    with pytest.raises(sv.SpecError):
        sv.spec_paged_attention(d["q"], d["start"], d["len"], d["tables"].t(), d["kp"], d["vp"], 2)
    odd = torch.zeros(2 * 8 * 64 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(2, 8, 64)
    with pytest.raises(sv.SpecError):
        sv.spec_paged_attention(odd, d["start"], d["len"], d["tables"], d["kp"], d["vp"], 2)
    k = torch.zeros((3, 2, 64), dtype=torch.bfloat16, device="cuda")
    for bad in (lambda: sv.spec_paged_append(k, k[:2], i32([0, 1, 2]), None, d["kp"], d["vp"]),
                lambda: sv.spec_paged_append(k, k, i32([0, 1]), None, d["kp"], d["vp"]),
                lambda: sv.spec_paged_append(k.half(), k, i32([0, 1, 2]), None, d["kp"], d["vp"]),
                lambda: sv.spec_paged_append(k, k, i32([0, 1, 2]), torch.zeros(1, device="cuda"), d["kp"], d["vp"]),
                lambda: sv.spec_pages_step(i32([0] * 12), i32([0] * 4), i32([0]), i32([0]), i32([0]), i32([0, 0]), i32([0])),
                lambda: sv.spec_pages_step(i32([0] * 12), i32([[0] * 4]), i32([0]), i32([0]), i32([0]), i32([0]), i32([0])),
                lambda: sv.spec_pages_init(i32([0] * 8))):
        with pytest.raises(sv.SpecError):
            bad()
