"""Cases of the paged-cache operators: page tables and slot maps stepped on the GPU, the
append that writes new keys and values at their slots, and the attention of each
sequence's new tokens over the pages.

With ``own`` false ``run`` computes the operators in elementary torch operations (32
bits, rounded once at the end); with ``own`` true it makes the framework's calls on the
same state.  Lengths follow from the case alone (``pattern`` seeds them), values and
page placement from the seed."""
import random

import torch

own = False

PAGE = 64          # positions per page
HEADER = 8         # int32 words in front of the free stack: [0] free pages, [1] error code


def listed():
    return [
        # one conversation growing by one token: the call's latency is all there is
        dict(name="pages: one sequence", op="pages", nseq=1, lo=100, hi=4000, add_lo=1, add_hi=1, crop=0, pattern=1),
        # a verify cycle of a full serving batch: rejected tails cropped, blocks of 8 added
        dict(name="pages: verify cycle of 200", op="pages", nseq=200, lo=1, hi=8000, add_lo=8, add_hi=8, crop=7, pattern=2),
        # prompts of many lengths admitted at once (their old pages released first)
        dict(name="pages: 1024 prompts", op="pages", nseq=1024, lo=1, hi=4000, add_lo=1, add_hi=4000, crop=4000, pattern=3),
        # decode append of a batch, keys and values cut from the fused QKV rows
        dict(name="append: 64 decode rows", op="append", rows=64, hq=32, hkv=8, hd=128, fused=True, pages=600, pattern=4),
        # prompt append of one long prompt
        dict(name="append: 16001 prompt rows", op="append", rows=16001, hq=32, hkv=8, hd=128, fused=True, pages=300, pattern=5),
        # narrow heads, rows contiguous
        dict(name="append: 777 rows of 4x64", op="append", rows=777, hq=4, hkv=4, hd=64, fused=False, pages=100, pattern=6),
        # the first tokens of one conversation (Llama-3.1-8B heads): latency
        dict(name="attn: 1 sequence of 300", op="attn", nseq=1, lo=300, hi=300, new_lo=1, new_hi=1, hq=32, hkv=8, hd=128, pattern=7),
        # the default verify block: 8 rows after 4096 positions
        dict(name="attn: verify 8 at 4104", op="attn", nseq=1, lo=4104, hi=4104, new_lo=8, new_hi=8, hq=32, hkv=8, hd=128, pattern=8),
        # one long document, one new token: all of the card on one sequence
        dict(name="attn: 1 sequence of 100003", op="attn", nseq=1, lo=100003, hi=100003, new_lo=1, new_hi=1, hq=32, hkv=8, hd=128, pattern=9),
        # decode of a ragged serving batch
        dict(name="attn: 64 ragged, decode", op="attn", nseq=64, lo=1, hi=8192, new_lo=1, new_hi=1, hq=32, hkv=8, hd=128, pattern=10),
        # ragged verify blocks over many short sequences, 64-wide heads, some slots idle
        dict(name="attn: 200 short, ragged blocks", op="attn", nseq=200, lo=16, hi=1500, new_lo=0, new_hi=8, hq=16, hkv=4, hd=64, pattern=11),
        # blocks of 16 with 8 query heads per kv head: 128 rows against each key
        dict(name="attn: 24 ragged, blocks of 16", op="attn", nseq=24, lo=500, hi=8000, new_lo=16, new_hi=16, hq=64, hkv=8, hd=128, pattern=12),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["pages", "append", "attn", "attn"])
    pattern = rng.randrange(1, 1 << 24)
    if op == "pages":
        nseq = _log_uniform(rng, 1, 1024)
        hi = _log_uniform(rng, 64, 4000)
        if rng.random() < 0.6:
            n = rng.randint(1, 16)
            return dict(op=op, nseq=nseq, lo=1, hi=hi, add_lo=n, add_hi=n, crop=n - 1, pattern=pattern)
        return dict(op=op, nseq=nseq, lo=1, hi=hi, add_lo=1, add_hi=_log_uniform(rng, 1, 4000), crop=hi, pattern=pattern)
    hd = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 5, 8, 16])
    if op == "append":
        g = rng.choice([1, 3, 4])
        rows = _log_uniform(rng, 1, 16000 * 8 // max(8, hkv))
        return dict(op=op, rows=rows, hq=g * hkv, hkv=hkv, hd=hd, fused=rng.random() < 0.5,
                    pages=(rows + PAGE - 1) // PAGE + _log_uniform(rng, 1, 300), pattern=pattern)
    g = rng.choice([1, 2, 3, 4, 4, 7, 8])
    nseq = _log_uniform(rng, 1, 200)
    hi = _log_uniform(rng, 32, 8192 if nseq > 4 else 100000)
    hi = max(32, min(hi, 64 * 5000 * 8 // (nseq * max(8, hkv))))
    n = rng.choice([1, 1, 2, 4, 8, 16])
    hi = max(32, min(hi, int(5e10 / (4 * nseq * n * g * hkv * hd))))
    ragged = rng.random() < 0.5
    return dict(op=op, nseq=nseq, lo=16 if ragged else max(16, hi // 2), hi=hi, new_lo=0 if ragged else n, new_hi=n,
                hq=g * hkv, hkv=hkv, hd=hd, pattern=pattern)


# ----------------------------------------------------------------- lengths --
def _lens(c):
    """Lengths of the case's sequences: pages (len, keep, add); attn (len, new)."""
    r = random.Random(c["pattern"])
    if c["op"] == "pages":
        out = []
        for _ in range(c["nseq"]):
            n = r.randint(c["lo"], c["hi"])
            out.append((n, n - min(n, r.randint(0, c["crop"])), r.randint(c["add_lo"], c["add_hi"])))
        return out
    out = []
    for _ in range(c["nseq"]):
        new = r.randint(c["new_lo"], c["new_hi"])
        out.append((max(new, r.randint(c["lo"], c["hi"])), new))
    return out if any(new for _, new in out) else [(max(1, n), 1) for n, _ in out]


def _pages(n):
    return (n + PAGE - 1) // PAGE


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _normal(shape, gen):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16)


def _tables(held, width, num_pages, gen):
    """Table [nseq][width] of distinct random pages (0 past the held ones) and the pages left over."""
    perm = torch.randperm(num_pages, generator=gen, device="cuda").to(torch.int32)
    held = torch.tensor(held, device="cuda")
    first = held.cumsum(0) - held
    j = torch.arange(width, device="cuda")
    at = (first[:, None] + j).clamp(max=num_pages - 1)
    zero = torch.zeros((), dtype=torch.int32, device="cuda")
    return torch.where(j < held[:, None], perm[at], zero).contiguous(), perm[int(held.sum()):]


# ----------------------------------------------------------------- prepare --
def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    if case["op"] == "pages":
        lens = _lens(case)
        held = [_pages(n) for n, _, _ in lens]
        need = [_pages(k + a) for _, k, a in lens]
        width = max(held + need)
        num_pages = sum(max(h, n) for h, n in zip(held, need)) + 64 + sum(held) // 8
        tables, free = _tables(held, width, num_pages, gen)
        pool = torch.zeros(HEADER + num_pages, dtype=torch.int32, device="cuda")
        pool[0] = free.numel()
        pool[HEADER:HEADER + free.numel()] = free
        rows = sum(a for _, _, a in lens)
        # every pass crops to keep and grows by add: from the second on the lengths stand at keep + add
        return dict(op="pages", pool=pool, tables=tables, len=_i32([n for n, _, _ in lens]), keep=_i32([k for _, k, _ in lens]),
                    add=_i32([a for _, _, a in lens]), row_start=torch.zeros(case["nseq"] + 1, dtype=torch.int32, device="cuda"),
                    slots=torch.full((rows,), -1, dtype=torch.int32, device="cuda"))
    hkv, hd, hq = case["hkv"], case["hd"], case["hq"]
    if case["op"] == "append":
        rows, pages = case["rows"], case["pages"]
        if case["fused"]:
            qkv = _normal((rows, (hq + 2 * hkv) * hd), gen)
            k = qkv[:, hq * hd:(hq + hkv) * hd].unflatten(1, (hkv, hd))
            v = qkv[:, (hq + hkv) * hd:].unflatten(1, (hkv, hd))
        else:
            k, v = _normal((rows, hkv, hd), gen), _normal((rows, hkv, hd), gen)
        if rows > 1000:   # a prompt: consecutive positions over shuffled pages
            perm = torch.randperm(pages, generator=gen, device="cuda")[:_pages(rows)]
            slots = (perm[:, None] * PAGE + torch.arange(PAGE, device="cuda")).reshape(-1)[:rows]
        else:             # single rows of many sequences
            slots = torch.randperm(pages * PAGE, generator=gen, device="cuda")[:rows]
        return dict(op="append", k=k, v=v, slots=slots.to(torch.int32), rows=_i32([rows]),
                    kpool=_normal((pages, hkv, PAGE, hd), gen), vpool=_normal((pages, hkv, PAGE, hd), gen))
    lens = _lens(case)
    held = [_pages(n) for n, _ in lens]
    width = max(held)
    num_pages = sum(held) + 1 + sum(held) // 8
    tables, _ = _tables(held, width, num_pages, gen)
    start = [0]
    for _, new in lens:
        start.append(start[-1] + new)
    # queries twice as long as unit keys make them: scores of a trained model's spread
    return dict(op="attn", q=2 * _normal((start[-1], hq, hd), gen), row_start=_i32(start), len=_i32([n for n, _ in lens]), tables=tables,
                kpool=_normal((num_pages, hkv, PAGE, hd), gen), vpool=_normal((num_pages, hkv, PAGE, hd), gen), max_new=max(new for _, new in lens))


# --------------------------------------------------------------------- run --
def run(state):
    if own:
        return _run_own(state)
    return {"pages": _plain_pages, "append": _plain_append, "attn": _plain_attn}[state["op"]](state)


def _run_own(s):
    import speculative_decoding_verify_pass_gb300 as sv
    if s["op"] == "pages":
        sv.spec_pages_step(s["pool"], s["tables"], s["len"], s["keep"], s["add"], s["row_start"], s["slots"])
        return dict(pool=s["pool"], tables=s["tables"], len=s["len"], row_start=s["row_start"], slots=s["slots"])
    if s["op"] == "append":
        sv.spec_paged_append(s["k"], s["v"], s["slots"], s["rows"], s["kpool"], s["vpool"])
        return dict(kpool=s["kpool"], vpool=s["vpool"])
    return sv.spec_paged_attention(s["q"], s["row_start"], s["len"], s["tables"], s["kpool"], s["vpool"], s["max_new"])


def _plain_pages(s):
    pool, tables, length, keep, add = s["pool"], s["tables"], s["len"], s["keep"], s["add"]
    nseq, width = tables.shape
    num_pages, rows = pool.numel() - HEADER, s["slots"].numel()
    new = keep + add
    held, need = (length + PAGE - 1) // PAGE, (new + PAGE - 1) // PAGE
    j = torch.arange(width, device=pool.device, dtype=torch.int32)
    gone = (j >= need[:, None]) & (j < held[:, None])
    come = (j >= held[:, None]) & (j < need[:, None])
    count, given, taken = pool[0].long(), gone.sum(), come.sum()
    ok = ((keep >= 0) & (keep <= length) & (add >= 0) & (need <= width)).all()
    ok = ok & (add.sum() <= rows) & (count + given <= num_pages) & (taken <= count + given)
    gone, come = gone & ok, come & ok
    # released pages go on the stack in (sequence, page) order; new ones come off its top
    stack = torch.cat([pool[HEADER:], pool.new_zeros(1)])
    to = torch.where(gone, count + gone.flatten().cumsum(0).view_as(gone) - 1, num_pages)
    stack[to] = torch.where(gone, tables, stack[num_pages])
    at = torch.where(come, count + given - come.flatten().cumsum(0).view_as(come), 0)
    tables.copy_(torch.where(come, stack[at], tables))
    pool[HEADER:] = stack[:num_pages]
    pool[0] = torch.where(ok, count + given - taken, count)
    length.copy_(torch.where(ok, new, length))
    s["row_start"][1:] = torch.where(ok, add.cumsum(0), 0)
    r = torch.arange(rows, device=pool.device, dtype=torch.int32)
    b = torch.searchsorted(s["row_start"][1:].contiguous(), r, right=True).clamp(max=nseq - 1)
    pos = keep[b] + r - s["row_start"][b]
    slot = tables[b, (pos // PAGE).clamp(0, width - 1).long()] * PAGE + pos % PAGE
    s["slots"].copy_(torch.where(r < s["row_start"][nseq], slot, s["slots"]))
    return dict(pool=pool, tables=tables, len=length, row_start=s["row_start"], slots=s["slots"])


def _plain_append(s):
    slot = s["slots"].long()
    s["kpool"][slot // PAGE, :, slot % PAGE] = s["k"]
    s["vpool"][slot // PAGE, :, slot % PAGE] = s["v"]
    return dict(kpool=s["kpool"], vpool=s["vpool"])


def _plain_attn(s):
    q, start, length, tables = s["q"], s["row_start"], s["len"], s["tables"]
    rows, hq, hd = q.shape
    nseq, width = tables.shape
    hkv, n, span = s["kpool"].shape[1], s["max_new"], width * PAGE
    g = hq // hkv
    pos = torch.arange(span, device=q.device)
    k = s["kpool"][tables.long()].transpose(1, 2).reshape(nseq, hkv, span, hd).float()
    v = s["vpool"][tables.long()].transpose(1, 2).reshape(nseq, hkv, span, hd).float()
    r = torch.arange(rows, device=q.device, dtype=torch.int32)
    b = torch.searchsorted(start[1:].contiguous(), r, right=True)
    j = (r - start[b]).long()
    block = torch.zeros(nseq, n, hq, hd, device=q.device)
    block[b, j] = q.float()
    block = block.view(nseq, n, hkv, g, hd).transpose(1, 2).reshape(nseq, hkv, n * g, hd)
    score = (block @ k.transpose(2, 3)).view(nseq, hkv, n, g, span) * hd ** -0.5
    last = (length - (start[1:] - start[:-1]))[:, None] + torch.arange(n, device=q.device)
    hidden = pos > last[:, None, :, None, None]
    score = score.masked_fill(hidden, float("-inf"))
    w = torch.exp(score - score.amax(-1, keepdim=True).clamp(min=-1e30)).view(nseq, hkv, n * g, span)
    o = (w @ v) / w.sum(-1, keepdim=True).clamp(min=1e-30)
    return o.view(nseq, hkv, n, g, hd).transpose(1, 2)[b, j].reshape(rows, hq, hd).to(q.dtype)


# -------------------------------------------------------------------- work --
def work(case):
    if case["op"] == "pages":
        lens = _lens(case)
        moved = sum(abs(_pages(k + a) - _pages(n)) for n, k, a in lens)
        rows = sum(a for _, _, a in lens)
        touched = sum(_pages(k + a) - k // PAGE for _, k, a in lens if a)
        return dict(bytes=4.0 * (5 * case["nseq"] + 2 * moved + rows + touched), flops=0.0)
    row = case["hkv"] * case["hd"] * 2.0
    if case["op"] == "append":
        return dict(bytes=case["rows"] * (4 * row + 4.0), flops=0.0)
    lens = [(n, new) for n, new in _lens(case) if new]
    new = sum(m for _, m in lens)
    seen = sum(m * (n - m) + m * (m + 1) // 2 for n, m in lens)
    return dict(bytes=sum(n for n, _ in lens) * 2 * row + new * case["hq"] * case["hd"] * 4.0 + sum(_pages(n) for n, _ in lens) * 4.0,
                flops=4.0 * seen * case["hq"] * case["hd"])


# ------------------------------------------------------------------- exact --
def exact(case, seed):
    """Definition in 64 bits, one sequence at a time; None where outputs are whole numbers."""
    if case["op"] == "pages":
        return None
    s = prepare(case, seed)
    if case["op"] == "append":
        out = {}
        for name, rows in (("kpool", s["k"]), ("vpool", s["v"])):
            flat = s[name].double().transpose(1, 2).reshape(-1, case["hkv"], case["hd"])
            flat[s["slots"].long()] = rows.double()
            out[name] = flat.view(-1, PAGE, case["hkv"], case["hd"]).transpose(1, 2).contiguous()
        return out
    g = case["hq"] // case["hkv"]
    start = s["row_start"].tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for i, (n, new) in enumerate(_lens(case)):
        pages = s["tables"][i, :_pages(n)].long()
        k = s["kpool"][pages].double().permute(1, 0, 2, 3).flatten(1, 2)[:, :n]
        v = s["vpool"][pages].double().permute(1, 0, 2, 3).flatten(1, 2)[:, :n]
        for a in range(new):
            seen = n - new + a + 1
            q = s["q"][start[i] + a].double().view(case["hkv"], g, case["hd"])
            w = torch.softmax(torch.matmul(q, k[:, :seen].transpose(1, 2)) / case["hd"] ** 0.5, -1)
            out[start[i] + a] = torch.matmul(w, v[:, :seen]).reshape(case["hq"], case["hd"])
    return out
