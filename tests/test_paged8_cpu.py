"""The 8-bit paged cache's argument checks, answered on the host before any CUDA
call: every refusal here uses pointers that are never followed."""
import ctypes

import pytest

P = 1 << 20        # a 256-byte aligned address that nothing dereferences


@pytest.fixture(scope="module")
def lib():
    import speculative_decoding_verify_pass_gb300 as sv
    from speculative_decoding_verify_pass_gb300 import _build
    _build.build()
    return sv.library()


def refused(lib, status, word, call):
    import speculative_decoding_verify_pass_gb300 as sv
    assert status == sv.SPEC_ERR_INVALID_ARG
    said = lib.spec_last_error().decode()
    assert word in said and said.startswith(call)


ROWS = dict(k=P, ks=512, v=P, vs=512, slots=P, count=None, rows=3, hkv=4, hd=128, kpool=P, vpool=P, scales=P, pages=8, err=None)


def append(lib, a):
    return lib.spec_paged_append_fp8(a["k"], a["ks"], a["v"], a["vs"], a["slots"], a["count"], a["rows"], a["hkv"], a["hd"], a["kpool"],
                                     a["vpool"], a["scales"], a["pages"], a["err"], None)


def read(lib, a):
    return lib.spec_paged_read_fp8(a["slots"], a["count"], a["rows"], a["hkv"], a["hd"], a["kpool"], a["vpool"], a["scales"], a["pages"],
                                   a["k"], a["ks"], a["v"], a["vs"], a["err"], None)


@pytest.mark.parametrize("call,name", [(append, "spec_paged_append_fp8"), (read, "spec_paged_read_fp8")])
@pytest.mark.parametrize("over,word", [
    (dict(k=None), "null"), (dict(v=None), "null"), (dict(slots=None), "null"), (dict(kpool=None), "null"), (dict(vpool=None), "null"),
    (dict(scales=None), "null"), (dict(rows=-1), "rows"), (dict(hd=96), "head_dim"), (dict(hkv=0), "n_kv_heads"),
    (dict(hkv=1025), "n_kv_heads"), (dict(pages=0), "num_pages"), (dict(pages=33554432), "num_pages"), (dict(ks=511), "strides"),
    (dict(ks=504), "strides"), (dict(vs=516), "strides"), (dict(vs=1 << 38), "strides"), (dict(k=P + 8), "aligned"),
    (dict(vpool=P + 2), "aligned"), (dict(scales=P + 8), "aligned"), (dict(slots=P + 2), "aligned"), (dict(count=P + 1), "aligned"),
    (dict(err=P + 3), "aligned")])
def test_append_and_read_refusals(lib, call, name, over, word):
    refused(lib, call(lib, dict(ROWS, **over)), word, name)


ATTN = dict(q=P, qs=1024, start=P, length=P, tables=P, width=40, nseq=2, rows=3, max_new=2, hq=8, hkv=2, hd=128, scale=0.1, kpool=P,
            vpool=P, scales=P, pages=8, out=P, os=1024, err=None, work=P, wbytes=1 << 30)


def attend(lib, a):
    return lib.spec_paged_attention_fp8(a["q"], a["qs"], a["start"], a["length"], a["tables"], a["width"], a["nseq"], a["rows"],
                                        a["max_new"], a["hq"], a["hkv"], a["hd"], a["scale"], a["kpool"], a["vpool"], a["scales"],
                                        a["pages"], a["out"], a["os"], a["err"], a["work"], a["wbytes"], None)


@pytest.mark.parametrize("over,word", [
    (dict(q=None), "null"), (dict(start=None), "null"), (dict(length=None), "null"), (dict(tables=None), "null"),
    (dict(kpool=None), "null"), (dict(vpool=None), "null"), (dict(scales=None), "null"), (dict(out=None), "null"),
    (dict(hd=32), "head_dim"), (dict(hq=9), "multiple"), (dict(hkv=0), "multiple"),
    (dict(hq=0), "multiple"), (dict(hq=129, hkv=1, qs=1 << 15, os=1 << 15), "128 query heads"), (dict(max_new=0), "max_new"),
    (dict(nseq=1025), "nseq"), (dict(nseq=-1), "nseq"), (dict(rows=-1), "rows"), (dict(width=0), "table_pages"),
    (dict(width=1 << 21), "table_pages"), (dict(pages=0), "num_pages"),
    (dict(pages=33554431, hkv=1024, hq=1024, qs=1 << 17, os=1 << 17), "fit int32"), (dict(scale=0.0), "scale"),
    (dict(scale=-1.0), "scale"), (dict(scale=float("nan")), "scale"), (dict(scale=float("inf")), "scale"), (dict(qs=1016), "strides"),
    (dict(os=1028), "strides"), (dict(q=P + 4), "aligned"), (dict(out=P + 8), "aligned"), (dict(kpool=P + 2), "aligned"),
    (dict(scales=P + 8), "aligned"), (dict(length=P + 2), "aligned"), (dict(err=P + 1), "aligned")])
def test_attention_refusals(lib, over, word):
    refused(lib, attend(lib, dict(ATTN, **over)), word, "spec_paged_attention_fp8")


def test_workspace_refusals(lib):
    out = ctypes.c_size_t(7)
    ask = lib.spec_paged_attention_fp8_workspace
    name = "spec_paged_attention_fp8"
    refused(lib, ask(8, 2, 128, 1, 40, None), "null", name)
    refused(lib, ask(8, 3, 128, 1, 40, ctypes.byref(out)), "multiple", name)
    refused(lib, ask(8, 2, 80, 1, 40, ctypes.byref(out)), "head_dim", name)
    refused(lib, ask(8, 2, 128, 0, 40, ctypes.byref(out)), "max_new", name)
    refused(lib, ask(8, 2, 128, 1, 0, ctypes.byref(out)), "table_pages", name)
    assert out.value == 7
    assert ask(8, 2, 128, 1, 16, ctypes.byref(out)) == 0 and out.value == 0


def test_nothing_to_do_is_no_error(lib):
    none = dict(k=None, v=None, slots=None, kpool=None, vpool=None, scales=None)
    assert append(lib, dict(ROWS, rows=0, **none)) == 0 and read(lib, dict(ROWS, rows=0, **none)) == 0
    none = dict(q=None, start=None, length=None, tables=None, kpool=None, vpool=None, scales=None, out=None, work=None, wbytes=0)
    assert attend(lib, dict(ATTN, nseq=0, **none)) == 0 and attend(lib, dict(ATTN, rows=0, **none)) == 0


def test_binding_refuses_host_tensors_and_wrong_types():
    torch = pytest.importorskip("torch")
    import speculative_decoding_verify_pass_gb300 as sv
    i = torch.zeros(16, dtype=torch.int32)
    t = torch.zeros((2, 4), dtype=torch.int32)
    pool = torch.zeros((3, 2, 64, 64), dtype=torch.float8_e4m3fn)
    scales = torch.zeros((3, 2, 2, 64), dtype=torch.uint8)
    rows = torch.zeros((2, 2, 64), dtype=torch.bfloat16)
    for call in (lambda: sv.spec_paged_append_fp8(rows, rows, i, None, pool, pool, scales),
                 lambda: sv.spec_paged_append_fp8(rows, rows, i, None, pool, pool, None),
                 lambda: sv.spec_paged_read_fp8(i, None, pool, pool, scales),
                 lambda: sv.spec_paged_attention_fp8(rows, i, i, t, pool, pool, scales, 1),
                 lambda: sv.spec_paged_attention_fp8(rows, i, i, t, pool, pool, None, 1)):
        with pytest.raises(sv.SpecError) as e:
            call()
        assert e.value.status == sv.SPEC_ERR_INVALID_ARG
