"""The paged-cache calls' argument checks, answered on the host before any CUDA
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


def refused(lib, status, word):
    import speculative_decoding_verify_pass_gb300 as sv
    assert status == sv.SPEC_ERR_INVALID_ARG
    assert word in lib.spec_last_error().decode()


@pytest.mark.parametrize("pool,pages,word", [(None, 4, "null"), (P + 1, 4, "aligned"), (P, 0, "num_pages"),
                                             (P, 33554432, "num_pages")])
def test_pages_init_refusals(lib, pool, pages, word):
    refused(lib, lib.spec_pages_init(pool, pages, None), word)


STEP = dict(pool=P, num_pages=8, tables=P, table_pages=4, length=P, keep=P, add=P, nseq=2, row_start=P, slots=P, row_cap=4)


@pytest.mark.parametrize("over,word", [
    (dict(pool=None), "null"), (dict(tables=None), "null"), (dict(length=None), "null"), (dict(keep=None), "null"),
    (dict(add=None), "null"), (dict(row_start=None), "null"), (dict(slots=None), "null"), (dict(nseq=-1), "nseq"),
    (dict(nseq=1025), "nseq"), (dict(num_pages=0), "num_pages"), (dict(num_pages=33554432), "num_pages"),
    (dict(table_pages=0), "table_pages"), (dict(table_pages=1048577), "table_pages"), (dict(row_cap=-1), "row_cap"),
    (dict(keep=P + 2), "aligned"), (dict(slots=P + 1), "aligned")])
def test_pages_step_refusals(lib, over, word):
    a = dict(STEP, **over)
    refused(lib, lib.spec_pages_step(a["pool"], a["num_pages"], a["tables"], a["table_pages"], a["length"], a["keep"],
                                     a["add"], a["nseq"], a["row_start"], a["slots"], a["row_cap"], None), word)


APPEND = dict(k=P, ks=512, v=P, vs=512, slots=P, count=None, rows=3, hkv=4, hd=128, kpool=P, vpool=P, pages=8, err=None)


@pytest.mark.parametrize("over,word", [
    (dict(k=None), "null"), (dict(v=None), "null"), (dict(slots=None), "null"), (dict(kpool=None), "null"),
    (dict(vpool=None), "null"), (dict(rows=-1), "rows"), (dict(hd=96), "head_dim"), (dict(hkv=0), "n_kv_heads"),
    (dict(hkv=1025), "n_kv_heads"), (dict(pages=0), "num_pages"), (dict(ks=511), "strides"), (dict(ks=504), "strides"),
    (dict(vs=516), "strides"), (dict(k=P + 8), "aligned"), (dict(vpool=P + 2), "aligned"), (dict(slots=P + 2), "aligned"),
    (dict(count=P + 1), "aligned"), (dict(err=P + 3), "aligned")])
def test_paged_append_refusals(lib, over, word):
    a = dict(APPEND, **over)
    refused(lib, lib.spec_paged_append(a["k"], a["ks"], a["v"], a["vs"], a["slots"], a["count"], a["rows"], a["hkv"],
                                       a["hd"], a["kpool"], a["vpool"], a["pages"], a["err"], None), word)


ATTN = dict(q=P, qs=1024, start=P, length=P, tables=P, width=40, nseq=2, rows=3, max_new=2, hq=8, hkv=2, hd=128,
            scale=0.1, kpool=P, vpool=P, pages=8, out=P, os=1024, err=None, work=P, wbytes=1 << 30)


@pytest.mark.parametrize("over,word", [
    (dict(q=None), "null"), (dict(start=None), "null"), (dict(length=None), "null"), (dict(tables=None), "null"),
    (dict(kpool=None), "null"), (dict(vpool=None), "null"), (dict(out=None), "null"), (dict(work=None), "null"),
    (dict(hd=32), "head_dim"), (dict(hq=9), "multiple"), (dict(hkv=0), "multiple"), (dict(hq=0), "multiple"),
    (dict(hq=129, hkv=1, qs=1 << 15, os=1 << 15), "128 query heads"), (dict(max_new=0), "max_new"), (dict(nseq=1025), "nseq"),
    (dict(nseq=-1), "nseq"), (dict(rows=-1), "rows"), (dict(width=0), "table_pages"), (dict(width=1 << 21), "table_pages"),
    (dict(pages=0), "num_pages"), (dict(pages=33554431, hkv=1024, hq=1024, qs=1 << 17, os=1 << 17), "fit int32"),
    (dict(scale=0.0), "scale"), (dict(scale=-1.0), "scale"), (dict(scale=float("nan")), "scale"),
    (dict(scale=float("inf")), "scale"), (dict(qs=1016), "strides"), (dict(os=1028), "strides"), (dict(q=P + 4), "aligned"),
    (dict(out=P + 8), "aligned"), (dict(kpool=P + 2), "aligned"), (dict(length=P + 2), "aligned"),
    (dict(err=P + 1), "aligned"), (dict(work=P + 16), "aligned"), (dict(wbytes=16), "work_bytes")])
def test_paged_attention_refusals(lib, over, word):
    a = dict(ATTN, **over)
    refused(lib, lib.spec_paged_attention(a["q"], a["qs"], a["start"], a["length"], a["tables"], a["width"], a["nseq"],
                                          a["rows"], a["max_new"], a["hq"], a["hkv"], a["hd"], a["scale"], a["kpool"],
                                          a["vpool"], a["pages"], a["out"], a["os"], a["err"], a["work"], a["wbytes"],
                                          None), word)


def test_paged_attention_workspace_refusals(lib):
    out = ctypes.c_size_t(7)
    refused(lib, lib.spec_paged_attention_workspace(8, 2, 128, 1, 40, None), "null")
    refused(lib, lib.spec_paged_attention_workspace(8, 3, 128, 1, 40, ctypes.byref(out)), "multiple")
    refused(lib, lib.spec_paged_attention_workspace(8, 2, 80, 1, 40, ctypes.byref(out)), "head_dim")
    refused(lib, lib.spec_paged_attention_workspace(8, 2, 128, 0, 40, ctypes.byref(out)), "max_new")
    refused(lib, lib.spec_paged_attention_workspace(8, 2, 128, 1, 0, ctypes.byref(out)), "table_pages")
    assert out.value == 7
    assert lib.spec_paged_attention_workspace(8, 2, 128, 1, 16, ctypes.byref(out)) == 0 and out.value == 0


def test_nothing_to_do_is_no_error(lib):
    assert lib.spec_pages_step(None, 8, None, 4, None, None, None, 0, None, None, 0, None) == 0
    assert lib.spec_paged_append(None, 512, None, 512, None, None, 0, 4, 128, None, None, 8, None, None) == 0
    assert lib.spec_paged_attention(None, 1024, None, None, None, 4, 0, 3, 1, 8, 2, 128, 0.1, None, None, 8, None, 1024,
                                    None, None, 0, None) == 0
    assert lib.spec_paged_attention(None, 1024, None, None, None, 4, 2, 0, 1, 8, 2, 128, 0.1, None, None, 8, None, 1024,
                                    None, None, 0, None) == 0


def test_binding_refuses_host_tensors_and_wrong_types():
    torch = pytest.importorskip("torch")
    import speculative_decoding_verify_pass_gb300 as sv
    i = torch.zeros(16, dtype=torch.int32)
    t = torch.zeros((2, 4), dtype=torch.int32)
    pool = torch.zeros((3, 2, 64, 64), dtype=torch.bfloat16)
    rows = torch.zeros((2, 2, 64), dtype=torch.bfloat16)
    for call in (lambda: sv.spec_pages_init(i), lambda: sv.spec_pages_step(i, t, i, i, i, i, i),
                 lambda: sv.spec_paged_append(rows, rows, i, None, pool, pool),
                 lambda: sv.spec_paged_attention(rows, i, i, t, pool, pool, 1)):
        with pytest.raises(sv.SpecError) as e:
            call()
        assert e.value.status == sv.SPEC_ERR_INVALID_ARG
