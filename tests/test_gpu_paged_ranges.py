"""Attention over the pages where its state moves: references that follow rising
scores over sums and outputs already formed, non-finite drafts on every tile and
over split pairs, batches too large for the lengths kept on chip, scores at the
ends of fp32.  The tolerance is test_gpu_paged's, computed here in 64 bits on the GPU."""
import random

import pytest

from gpu_common import torch_cuda
from test_gpu_paged import PAGE, Case, i32, pages_of, sv_

pytestmark = pytest.mark.gpu

CHUNK, WHOLE_PAGES = 128, 16
# (query heads per kv head, new rows): tiles of 16, 32, 64 and 128 rows, one of each kind not full
TILES = [(4, 1), (4, 4), (2, 12), (4, 8), (3, 16), (4, 16), (7, 16), (8, 16)]
TILE_OF = {(4, 1): 16, (4, 4): 16, (2, 12): 32, (4, 8): 32, (3, 16): 64, (4, 16): 64, (7, 16): 128, (8, 16): 128}


def scores(c, q, scale):
    """(scaled scores, their magnitudes summed) [kv head][row * group + g][position] of sequence q in 64 bits."""
    torch = torch_cuda()
    G, m = c.hq // c.hkv, c.new[q]
    x = c.q[c.start[q]:c.start[q] + m].cuda().double().view(m, c.hkv, G, c.hd).transpose(0, 1).reshape(c.hkv, m * G, c.hd)
    k = c.k[q].cuda().double().permute(1, 2, 0)
    return torch.matmul(x, k) * scale, torch.matmul(x.abs(), k.abs()) * scale


def visible(c, q):
    """[row * group + g][position]: whether the row sees the position."""
    torch = torch_cuda()
    n, m, G = c.lens[q], c.new[q], c.hq // c.hkv
    last = (n - m + torch.arange(m, device="cuda")).repeat_interleave(G)
    return torch.arange(n, device="cuda") <= last[:, None]


def reference(c, scale=None):
    """(out, bound) [rows][heads][dims] in 64 bits; the case's values have to be finite."""
    torch = torch_cuda()
    scale = c.hd ** -0.5 if scale is None else scale
    out = torch.zeros((c.rows, c.hq, c.hd), dtype=torch.float64, device="cuda")
    bound = torch.zeros_like(out)
    G = c.hq // c.hkv
    for q, (n, m) in enumerate(zip(c.lens, c.new)):
        if n == 0 or m == 0:
            continue
        s, a = scores(c, q, scale)
        see = visible(c, q)
        s, a = s.masked_fill(~see, -float("inf")), a.masked_fill(~see, 0.0)
        w = torch.exp(s - s.amax(-1, keepdim=True).clamp(min=-1e300))
        w = w / w.sum(-1, keepdim=True).clamp(min=1e-300)
        v = c.v[q].cuda().double().transpose(0, 1)
        d = (c.hd * 2.0 ** -24 * a + 2.0 ** -23 * s.masked_fill(~see, 0.0).abs()).amax(-1, keepdim=True)
        E = 2.0 ** -16 + 2.0 ** -21 + 4 * d + 2 * see.sum(-1)[None, :, None] * 2.0 ** -24
        o, ov = torch.matmul(w, v), torch.matmul(w, v.abs())

        def rows(x):
            return x.view(c.hkv, m, G, c.hd).transpose(0, 1).reshape(m, c.hq, c.hd)
        out[c.start[q]:c.start[q] + m] = rows(o)
        bound[c.start[q]:c.start[q] + m] = rows(2.0 ** -8 * o.abs() + E * (1 + 2.0 ** -8) * ov)
    return out, bound


def check(c, got, ref=None, rows=None, dims=None):
    out, bound = ref or reference(c)
    over = (got.double() - out).abs() - bound
    over = over[:c.start[-1]] if rows is None else over[rows]
    if dims is not None:
        over = over[:, :, dims]
    assert bool((over <= 0).all()), float(over.nan_to_num(nan=float("inf")).max())   # a NaN is not <= 0


def width(c, pages):
    """The case with tables of that many pages (all that it holds, at least)."""
    torch = torch_cuda()
    t = torch.full((len(c.lens), pages), 2 ** 31 - 1, dtype=torch.int32)
    have = min(pages, c.tables_cpu.shape[1])
    assert have >= max(pages_of(n) for n in c.lens)
    t[:, :have] = c.tables_cpu[:, :have]
    c.tables_cpu = t
    c.d["tables"] = t.cuda()
    return c


def repage(c):
    """Keys and values of the case written to its pages again."""
    torch = torch_cuda()
    for q, n in enumerate(c.lens):
        pages = c.tables_cpu[q, :pages_of(n)].long().cuda()
        for name, rows in (("kp", c.k[q]), ("vp", c.v[q])):
            pad = torch.full((pages.numel() * PAGE, c.hkv, c.hd), float("nan"), dtype=torch.bfloat16)
            pad[:n] = rows
            c.d[name][pages] = pad.view(-1, PAGE, c.hkv, c.hd).transpose(1, 2).contiguous().cuda()


def segments(c, tile, sms):
    """The CTAs' segments, from the deal's definition: (sequence, row block, kv head, first chunk, end chunk)."""
    G, whole = c.hq // c.hkv, c.tables_cpu.shape[1] <= WHOLE_PAGES
    tokens = tile // G
    pairs, at = [], 0
    for q, (n, m) in enumerate(zip(c.lens, c.new)):
        chunks = max(1, -(-n // CHUNK))
        for b in range(-(-m // tokens)):
            for h in range(c.hkv):
                pairs.append((at, at + chunks, q, b, h))
                at += chunks
    if whole:
        return [(q, b, h, 0, e - a) for a, e, q, b, h in pairs]
    work = min(at, sms)
    edges = [i * (at // work) + min(i, at % work) for i in range(work + 1)]
    out = []
    for lo, hi in zip(edges, edges[1:]):
        out += [(q, b, h, max(lo, a) - a, min(hi, e) - a) for a, e, q, b, h in pairs if a < hi and e > lo]
    return out


def moves_over_sums(c, tile):
    """How often a reference moves in a chunk that is not its first (then sums and outputs
    formed before have to move with it), by the kernel's rule: a group's reference is its first
    chunk's first key, and rises to a chunk's maximum where that exceeds it by more than 40 in
    log2 units.  Up to 64 rows alternate chunks of a segment belong to two groups."""
    torch = torch_cuda()
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    G = c.hq // c.hkv
    tokens, groups, count = tile // G, 2 if tile <= 64 else 1, 0
    tops = {}
    for q in range(len(c.lens)):
        s = scores(c, q, c.hd ** -0.5)[0].masked_fill(~visible(c, q), -float("inf")) * 1.4426950408889634
        pad = torch.full((s.shape[0], s.shape[1], -(-s.shape[2] // CHUNK) * CHUNK), -float("inf"), dtype=s.dtype, device="cuda")
        pad[:, :, :s.shape[2]] = s
        pad = pad.view(s.shape[0], s.shape[1], -1, CHUNK)
        tops[q] = pad[..., 0].cpu().numpy(), pad.amax(-1).cpu().numpy()
    for q, b, h, c0, c1 in segments(c, tile, sms):
        first, top = tops[q]
        r = slice(b * tokens * G, min(c.new[q], (b + 1) * tokens) * G)
        for g in range(groups):
            ref = None
            for k in range(c0 + g, c1, groups):
                if ref is None:
                    ref = first[h, r, k].clip(min=-1e30)
                    live = False
                if ((top[h, r, k] - ref) > 40.5).any():
                    ref = ref.clip(min=top[h, r, k])
                    count += live
                live = True
    return count


def rising(lens, new, heads, seed):
    """A case whose chunks reach 0, 43 and 86 (log2) above the other keys' scores, each level
    twice in a row, at a key in the middle of the chunk, with values as much smaller: what every
    level leaves in the result is of one size, and losing or keeping any shows."""
    hq, hkv, hd = heads
    torch = torch_cuda()
    c = Case(lens, new, hq, hkv, hd, seed=seed, qscale=1.0)
    c.q[:, :, 0] = 8.0
    c.d["q"].copy_(c.q)
    for q, n in enumerate(lens):
        t = torch.arange(n)
        level = 43.0 * ((t // CHUNK) % 6 // 2) * (t % CHUNK == 77)
        unit = 1.4426950408889634 * hd ** -0.5 * 8.0
        c.k[q][:, :, 0] = (level / unit).bfloat16()[:, None]
        c.v[q] = (c.v[q].float() * torch.exp2(40.0 - level)[:, None, None]).bfloat16()
    repage(c)
    return c


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("tile", TILES, ids=lambda t: "%dx%d" % t)
@pytest.mark.parametrize("split", [False, True], ids=["whole", "split"])
def test_references_that_rise_over_sums_and_outputs(tile, hd, split):
    group, m = tile
    if split:
        lens, hkv = [4210 + 7 * i for i in range(10)], 4
    else:
        lens, hkv = [1010, 897, 700], 2
    c = rising(lens, [m, max(1, m - 1), m] + [m] * (len(lens) - 3), (hkv * group, hkv, hd), seed=30)
    if not split:
        width(c, WHOLE_PAGES)
    assert moves_over_sums(c, TILE_OF[tile]) >= len(lens) * hkv
    check(c, c.run(max_new=m))


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("tile", TILES, ids=lambda t: "%dx%d" % t)
@pytest.mark.parametrize("n", [100, 129, 960, 1090, 1154, 1153, 2210])
def test_nonfinite_drafts_on_every_tile(tile, hd, n):
    """Drafted positions with a non-finite value or key, of which only later rows of the block
    know: on either page of the last chunk, over a chunk's border, pairs whole and split."""
    torch = torch_cuda()
    group, m = tile
    m = max(m, 3)                                      # of a tile for max_new rows, as many as needed
    hkv = 3
    for lens, new in (([n], [m]), ([n, 70, n + 1, 1300], [m, 2, m, 1])):
        c = Case(lens, new, hkv * group, hkv, hd, seed=n + hd, qscale=1.0)
        if n < 1000 and len(lens) == 1:
            width(c, WHOLE_PAGES)
        ref = reference(c)
        last = [float("nan"), float("inf"), -float("inf")]
        first_bad = {}
        for q in (0, 2) if len(lens) > 2 else (0,):
            for i, back in enumerate((2, 1)):          # the last two positions, a dimension each
                v = c.v[q][lens[q] - back].clone()
                v[:, 5 + 17 * i] = last[(q + i) % 3]
                c.put(q, lens[q] - back, v=v)
            first_bad[q] = c.start[q] + new[q] - 2
        got = c.run(max_new=tile[1])
        other = [d for d in range(hd) if d not in (5, 22)]
        clean = [r for q in range(len(lens)) for r in range(c.start[q], c.start[q + 1] if q not in first_bad else first_bad[q])]
        check(c, got, ref, rows=clean)
        check(c, got, ref, dims=other)
        for q, r in first_bad.items():
            assert not torch.isfinite(got[r:r + 2, :, 5]).any()
            assert torch.isfinite(got[r, :, 22]).all() and not torch.isfinite(got[r + 1, :, 22]).any()
        # a key that is not finite, seen by the last row alone
        c = Case(lens, new, hkv * group, hkv, hd, seed=n + hd, qscale=1.0)
        if n < 1000 and len(lens) == 1:
            width(c, WHOLE_PAGES)
        c.put(0, n - 1, k=torch.full((hkv, hd), last[n % 3]).bfloat16())
        got = c.run(max_new=tile[1])
        check(c, got, ref, rows=[r for r in range(c.start[-1]) if r != m - 1])


def test_nonfinite_values_of_a_prompt_cost_little():
    """A prompt whose last values are not finite, in every head: the blocks before them hide them and
    need no look at each of the positions behind (which took a hundred times the call's time)."""
    torch = torch_cuda()
    n, hq, hkv, hd = 6000, 32, 8, 128
    g = torch.Generator(device="cuda").manual_seed(7)
    pages = pages_of(n)
    q = torch.randn((n, hq, hd), generator=g, device="cuda").bfloat16()
    kp = torch.randn((pages, hkv, PAGE, hd), generator=g, device="cuda").bfloat16()
    vp = torch.randn((pages, hkv, PAGE, hd), generator=g, device="cuda").bfloat16()
    tables = torch.arange(pages, device="cuda", dtype=torch.int32)[None]
    start, length = i32([0, n]), i32([n])

    def run():
        return sv_().spec_paged_attention(q, start, length, tables, kp, vp, n)

    def timed():
        best = float("inf")
        for _ in range(4):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            run()
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b))
        return best
    clean, t_clean = run(), timed()
    vp[(n - 2) // PAGE, :, (n - 2) % PAGE:(n - 1) % PAGE + 1] = float("nan")
    got, t_nan = run(), timed()
    assert torch.equal(got[:n - 2].view(torch.int16), clean[:n - 2].view(torch.int16))
    assert got[n - 2:].isnan().all()
    assert t_nan < 4 * t_clean, (t_nan, t_clean)


@pytest.mark.parametrize("nseq", [64, 65, 200, 1024])
@pytest.mark.parametrize("heads", [(8, 2, 64), (8, 1, 128)])
def test_split_batches_around_the_lengths_kept_on_chip(nseq, heads):
    """Lengths are read from memory above 64 sequences; tables of more than 16 pages, so pairs are
    split and joined; idle, empty and long sequences among them."""
    rng = random.Random(nseq)
    lens = [rng.choice([0, 1, 64, 130, rng.randint(1, 1500)]) if nseq < 1000 else rng.choice([0, 3, 65, 300]) for _ in range(nseq)]
    lens[-1], lens[nseq // 2] = 2100, 1700
    new = [rng.randint(0, min(n, 5)) if n else rng.choice([0, 0, 2]) for n in lens]
    new[-1] = 3
    c = Case(lens, new, *heads, seed=nseq + heads[0], qscale=1.5)
    assert c.tables_cpu.shape[1] > WHOLE_PAGES
    err = i32([0])
    got = c.run(d_error=err)
    assert err.item() == 0
    check(c, got)


@pytest.mark.parametrize("sign", [1, -1], ids=["high", "low"])
@pytest.mark.parametrize("exponent", [14, 15, 17, 30, 50, 60])
@pytest.mark.parametrize("heads,lens,new", [((4, 2, 128), [700], [2]), ((8, 1, 64), [130, 5000], [16, 4]), ((4, 4, 64), [6000, 1, 64], [1, 1, 2]),
                                            ((16, 2, 128), [2600, 300], [16, 3]), ((12, 3, 64), [900, 250], [16, 5])])
def test_scores_of_any_size(sign, exponent, heads, lens, new):
    """Scores of +-2^30 to +-2^125, whose steps in fp32 reach far past the softmax's range: one key
    (or two equal ones) has all of the weight, and the result is its value (the mean of two), exactly."""
    torch = torch_cuda()
    hq, hkv, hd = heads
    c = Case(lens, new, hq, hkv, hd, seed=40)
    g = torch.Generator().manual_seed(exponent)
    c.q.zero_()
    c.q[:, :, 0] = 2.0 ** exponent
    c.d["q"].copy_(c.q)
    want = torch.zeros((c.rows, hq, hd), dtype=torch.float64)
    for q, (n, m) in enumerate(zip(lens, new)):
        times = torch.randint(5, 30, (n, hkv), generator=g).double()
        for h in range(hkv):
            seen = max(1, n - m + 1)                   # what all rows of the block see
            at = random.Random(h * 7 + q).sample(range(seen), min(seen, 1 + h % 2))
            times[at, h] = 30.0 if sign > 0 else 4.0
            o = torch.stack([c.v[q][t, h].double() for t in at]).mean(0)
            want[c.start[q]:c.start[q + 1], h * (hq // hkv):(h + 1) * (hq // hkv)] = o
        c.k[q][:, :, 0] = (sign * times * 2.0 ** exponent).bfloat16()
    repage(c)
    got = c.run(scale=1.0)
    assert torch.equal(got.cpu(), want.bfloat16())
