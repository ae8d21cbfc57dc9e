"""Rotary positions on the GPU against 64 bits.

Tolerance, per element: half a step of the result's type (eps / 2 of its value),
half a step of that type's smallest number, and E * g (|u| + |v|) for 32 bits: cos
and sin as sincospi gives them (2^-22 absolute: its error and that of its
argument, 24 bits of half a circle, 2^-24 pi), their product with the gain (2^-24),
two products and a sum (3 * 2^-24): E = 2^-21."""
import math

import numpy as np
import pytest

from gpu_common import torch_cuda

pytestmark = pytest.mark.gpu


def sv_():
    import speculative_decoding_verify_pass_gb300 as sv
    return sv


def i32(x):
    return torch_cuda().tensor(x, dtype=torch_cuda().int32, device="cuda")


def turned(x, pos, freq, gain, inter, inverse):
    """(definition in 64 bits, u and v magnitudes) of x [rows][heads][hd] (numpy float64)."""
    n = len(freq)
    a = np.asarray(pos, dtype=np.float64)[:, None, None] * np.asarray(freq) * (-1.0 if inverse else 1.0)
    at = np.arange(n) * 2 if inter else np.arange(n)
    to = at + 1 if inter else at + n
    u, v = x[..., at], x[..., to]
    out, size = x.copy(), np.zeros_like(x)
    out[..., at] = gain * (u * np.cos(a) - v * np.sin(a))
    out[..., to] = gain * (v * np.cos(a) + u * np.sin(a))
    size[..., at] = size[..., to] = abs(gain) * (np.abs(u) + np.abs(v))
    return out, size


def check(got, x, pos, freq, gain, inter, inverse):
    torch = torch_cuda()
    f = torch.finfo(got.dtype)
    want, size = turned(x.double().cpu().numpy(), pos, freq, gain, inter, inverse)
    g = got.double().cpu().numpy()
    bound = f.eps / 2 * np.abs(want) + f.tiny * f.eps / 2 + (1 + f.eps) * 2.0 ** -21 * size
    assert np.all(np.abs(g - want) <= bound), float((np.abs(g - want) - bound).max())
    n = len(freq)
    assert torch.equal(got[..., 2 * n:], x[..., 2 * n:])


def frequencies(turns):
    return turns.cpu().numpy().view(np.uint64).astype(np.float64) * 2.0 ** -64 * 2 * math.pi


@pytest.mark.parametrize("type", ["bfloat16", "float16", "float32"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("heads,hd,rot", [(1, 8, 2), (5, 64, 64), (40, 128, 128), (3, 128, 24), (7, 64, 22), (2, 256, 8), (1, 1024, 1024), (9, 72, 40)])
def test_matches_64_bits(type, inter, heads, hd, rot):
    torch = torch_cuda()
    sv = sv_()
    torch.manual_seed(heads + hd + rot)
    turns, gain = sv.spec_rope_table(rot, 1e4)
    freq = frequencies(turns)
    for rows, inverse, g in ((1, False, 1.0), (9, True, 1.0), (700, False, 1.25)):
        x = torch.randn((rows, heads, hd), device="cuda").to(getattr(torch, type))
        pos = torch.randint(0, 5000, (rows,), dtype=torch.int32, device="cuda")
        got = sv.spec_rope(x, turns, d_pos=pos, interleaved=inter, inverse=inverse, gain=g)
        check(got, x, pos.tolist(), freq, g, inter, inverse)


@pytest.mark.parametrize("pos", [0, 1, 65535, 10 ** 6 + 1, 2 ** 31 - 1, -1, -2 ** 31])
def test_far_positions(pos):
    """The angle is as exact at position 2^31 as at 1 (its fp64 value here is off by 2^-22 there: the frequency is taken as the table's)."""
    torch = torch_cuda()
    sv = sv_()
    turns, gain = sv.spec_rope_table(64, 5e5, sv.SPEC_ROPE_WAVELENGTH, 8.0)
    x = torch.randn((2, 3, 64), device="cuda")
    got = sv.spec_rope(x, turns, d_pos=i32([pos, pos]))
    t = [int(v) for v in turns.cpu().numpy().view(np.uint64)]
    # the angle within one circle, exactly, as a frequency at position 1
    freq = [(pos * v % 2 ** 64) / 2.0 ** 64 * 2 * math.pi for v in t]
    check(got, x, [1, 1], freq, 1.0, False, False)


@pytest.mark.parametrize("lens,new", [([7], [7]), ([100, 0, 5, 3000], [1, 0, 5, 16]), ([3] * 40, [0, 1, 3, 2] * 10), ([2], [5]),
                                      ([9] * 1024, [1] * 1024), ([2000], [700])])
def test_positions_of_each_sequences_newest_rows(lens, new):
    torch = torch_cuda()
    sv = sv_()
    start = [0]
    for m in new:
        start.append(start[-1] + m)
    rows = start[-1] + 3
    pos = [n - m + j for n, m in zip(lens, new) for j in range(m)]
    x = torch.randn((rows, 4, 64), device="cuda").bfloat16()
    turns, gain = sv.spec_rope_table(64, 1e4, sv.SPEC_ROPE_PARTS, 4.0)
    out = torch.full_like(x, 7.0)
    assert sv.spec_rope(x, turns, i32(start), i32(lens), gain=gain, d_out=out) is out
    check(out[:start[-1]], x[:start[-1]], pos, frequencies(turns), gain, False, False)
    assert (out[start[-1]:] == 7.0).all()
    same = x.clone()
    sv.spec_rope(same, turns, i32(start), i32(lens), gain=gain, d_out=same)
    assert torch.equal(same[:start[-1]], out[:start[-1]]) and torch.equal(same[start[-1]:], x[start[-1]:])


def test_bad_row_starts_and_lengths_stay_in_bounds():
    """Row starts that fall, lie outside or are all the same: nothing outside the rows is touched."""
    torch = torch_cuda()
    sv = sv_()
    turns, _ = sv.spec_rope_table(64)
    x = torch.randn((6, 2, 64), device="cuda")
    room = torch.full((10, 2, 64), 5.0, device="cuda")
    for start in ([0, 6, 3, 6], [-7, -3, 2, 9], [9, 9, 9, 9], [2 ** 31 - 1, 0, -2 ** 31, 5], [6, 5, 4, 3]):
        sv.spec_rope(x, turns, i32(start), i32([2 ** 31 - 1, -2 ** 31, 0]), d_out=room[2:8])
    assert (room[:2] == 5.0).all() and (room[8:] == 5.0).all()


@pytest.mark.parametrize("inter", [False, True])
def test_inverse_undoes_and_is_the_gradient(inter):
    torch = torch_cuda()
    sv = sv_()
    turns, _ = sv.spec_rope_table(48)
    x = torch.randn((20, 3, 64), device="cuda")
    w = torch.randn((20, 3, 64), device="cuda")
    pos = torch.arange(20, dtype=torch.int32, device="cuda") * 37
    there = sv.spec_rope(x, turns, d_pos=pos, interleaved=inter, gain=1.5)
    back = sv.spec_rope(there, turns, d_pos=pos, interleaved=inter, inverse=True, gain=1 / 1.5)
    # two calls' E = 2^-21 of (|u| + |v|), the first one's through the second's (|u| + |v|) again
    n = 24
    size = (x[..., 0:48:2].abs() + x[..., 1:48:2].abs()) if inter else (x[..., :n].abs() + x[..., n:48].abs())
    assert (back - x).abs()[..., :48].max().item() <= 4 * 2.0 ** -21 * size.max().item()
    # the gradient of sum(w * turned(x)) with the gain: turned back with the same gain.
    # (the tolerance is that of either side's 2^-21 (|u| + |v|) per element, over 64 * 3 * 20 products)
    grad = sv.spec_rope(w, turns, d_pos=pos, interleaved=inter, inverse=True, gain=1.5)
    tail = torch.ones(64, device="cuda")
    tail[48:] = 0
    a = (w * there * tail).double().sum().item()
    b = (grad * x * tail).double().sum().item()
    bound = 2 * 1.5 * 2.0 ** -21 * 2 * float((w.abs().max() * x.abs().max()).item()) * x.numel()
    assert abs(a - b) <= bound
    # and against a difference: the call is linear in x, so a step of one element is exact to rounding
    step = torch.zeros_like(x)
    step[3, 1, 5] = 1.0
    d = (sv.spec_rope(step, turns, d_pos=pos, interleaved=inter, gain=1.5) * w).double().sum().item()
    assert abs(d - grad[3, 1, 5].item()) <= 1e-5 * (1 + abs(d))


def test_strides_and_neighbours():
    """The queries and keys of fused QKV rows turned in place: the values beside them stay."""
    torch = torch_cuda()
    sv = sv_()
    qkv = torch.randn((33, 6, 128), device="cuda").bfloat16()
    keep = qkv.clone()
    turns, _ = sv.spec_rope_table(128, 5e5)
    pos = torch.arange(33, dtype=torch.int32, device="cuda")
    sv.spec_rope(qkv[:, :5], turns, d_pos=pos, d_out=qkv[:, :5])
    assert torch.equal(qkv[:, 5], keep[:, 5])
    check(qkv[:, :5], keep[:, :5], pos.tolist(), frequencies(turns), 1.0, False, False)


def test_graph_other_stream_and_refusals():
    torch = torch_cuda()
    sv = sv_()
    turns, _ = sv.spec_rope_table(64)
    x = torch.randn((5, 2, 64), device="cuda").bfloat16()
    start, length, out = i32([0, 5]), i32([5]), torch.empty_like(x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sv.spec_rope(x, turns, start, length, d_out=out)
    for n in (5, 900, 70000):
        length.fill_(n)
        g.replay()
        torch.cuda.synchronize()
        check(out, x, range(n - 5, n), frequencies(turns), 1.0, False, False)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = sv.spec_rope(x, turns, start, length)
    s.synchronize()
    assert torch.equal(other, out)
    p = i32([0] * 5)
    for bad in (lambda: sv.spec_rope(x, turns, start, length, d_pos=p), lambda: sv.spec_rope(x, turns),
                lambda: sv.spec_rope(x, turns, start), lambda: sv.spec_rope(x, turns, d_pos=p[:4]),
                lambda: sv.spec_rope(x, turns, start[:1], length), lambda: sv.spec_rope(x, turns.int(), d_pos=p),
                lambda: sv.spec_rope(x.double(), turns, d_pos=p), lambda: sv.spec_rope(x, turns, d_pos=p.long()),
                lambda: sv.spec_rope(x, turns, d_pos=p, d_out=x.float()), lambda: sv.spec_rope(x[..., :62], turns, d_pos=p),
                lambda: sv.spec_rope(x.transpose(1, 2), turns, d_pos=p), lambda: sv.spec_rope(x, turns.cpu(), d_pos=p),
                lambda: sv.spec_rope(x[:, :, :56].contiguous(), turns, d_pos=p), lambda: sv.spec_rope(x, turns, d_pos=p, gain=float("nan")),
                lambda: sv.spec_rope(x[:1].expand(5, 2, 64), turns, d_pos=p, d_out=x[:1].expand(5, 2, 64))):
        with pytest.raises(sv.SpecError):
            bad()
    assert sv.spec_rope(x[:0], turns, d_pos=p[:0]).shape == (0, 2, 64)


def test_a_batch_of_no_sequences():
    torch = torch_cuda()
    sv = sv_()
    turns, _ = sv.spec_rope_table(64)
    x, out = torch.randn((5, 3, 64), device="cuda").bfloat16(), torch.full((5, 3, 64), 7.0, device="cuda").bfloat16()
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    assert sv.spec_rope(x, turns, i32([0]), none, d_out=out) is out
    assert (out == 7.0).all()
    assert sv.spec_rope(x, turns, i32([0]), none).shape == x.shape


@pytest.mark.parametrize("over", [-1, 0, 1])
def test_rows_on_both_sides_of_where_a_row_gets_one_warp(over):
    """Up to 4 rows an SM of the device have 8 warps each."""
    torch = torch_cuda()
    sv = sv_()
    rows = 4 * torch.cuda.get_device_properties(0).multi_processor_count + over
    turns, _ = sv.spec_rope_table(48, 1e4)
    x = torch.randn((rows, 9, 64), device="cuda").bfloat16()
    pos = torch.randint(0, 100000, (rows,), dtype=torch.int32, device="cuda")
    check(sv.spec_rope(x, turns, d_pos=pos), x, pos.tolist(), frequencies(turns), 1.0, False, False)
