"""The serving operators without a GPU: refusals through the C ABI and the torch layer,
and the tests' own 64-bit restatements against hand-worked values."""

import math
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

import kv4_ref as R
from tiled_attention_tmem_gb300 import api, binding as b, build, serving

A = 1 << 20  # an aligned fake address; never dereferenced


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build_library()
    return b.lib()


def test_page_validation():
    ok = dict(B=2, width=4, page=16, T=8, free_size=9, lengths=A, new=A, table=A, free=A, count=A, slots=A, cu=A,
              held=A, out=A)

    def grow(**kw):
        a = {**ok, **kw}
        return b.fa_page_grow(a["lengths"], a["new"], a["table"], a["B"], a["width"], a["page"], a["free"],
                              a["free_size"], a["count"], a["T"], a["slots"], a["cu"], a["held"], a["out"], None)

    def slots(**kw):
        a = {**ok, **kw}
        return b.fa_page_slots(a["lengths"], a["new"], a["table"], a["B"], a["width"], a["page"], a["T"], a["slots"],
                               a["cu"], None)

    for call in (grow, slots):
        for bad in (dict(B=-1), dict(width=-1), dict(T=-1), dict(page=0), dict(page=24), dict(page=256),
                    dict(B=(1 << 21) + 1), dict(width=1 << 27), dict(lengths=0), dict(new=0), dict(table=0),
                    dict(slots=0), dict(cu=0)):
            assert call(**bad) == b.FA_ERR_INVALID_ARG, bad
        assert call(B=0, lengths=0, new=0, table=0, slots=0, cu=0) == b.FA_OK
    for bad in (dict(free=0), dict(count=0), dict(held=0), dict(out=0), dict(free_size=-1)):
        assert grow(**bad) == b.FA_ERR_INVALID_ARG, bad


def cache(a):
    c = b.FaKv4Cache(a["kc"], a["ks"], a["vc"], a["vs"], a["pages"], a["page"], a["H"], a["d"], a["kg"], a["vg"])
    KEEP.append(c)
    return c


KEEP = []


def test_store_and_load_validation():
    ok = dict(k=A, v=A, kt=256, kh=128, vt=256, vh=128, slots=A, T=4, H=2, d=128, kc=A, ks=A, vc=A, vs=A, pages=3,
              page=16, kg=1.0, vg=1.0)

    assert b.fa_kv4_store(None, A, A, 0, 0, 0, 0, A, 1, None) == b.FA_ERR_INVALID_ARG
    assert b.fa_kv4_load(None, A, 1, A, A, None) == b.FA_ERR_INVALID_ARG

    def store(**kw):
        a = {**ok, **kw}
        return b.fa_kv4_store(cache(a).address, a["k"], a["v"], a["kt"], a["kh"], a["vt"], a["vh"], a["slots"],
                              a["T"], None)

    def load(**kw):
        a = {**ok, **kw}
        return b.fa_kv4_load(cache(a).address, a["slots"], a["T"], a["k"], a["v"], None)

    for call in (store, load):
        for bad in (dict(T=-1), dict(H=-1), dict(pages=-1), dict(page=48), dict(kg=0.0), dict(vg=-1.0),
                    dict(kg=float("nan")), dict(vg=float("inf")), dict(kg=1e-45), dict(k=0), dict(v=0), dict(slots=0),
                    dict(kc=0), dict(vs=0)):
            assert call(**bad) == b.FA_ERR_INVALID_ARG, bad
        for bad in (dict(d=80), dict(d=32), dict(d=512)):
            assert call(**bad) == b.FA_ERR_UNSUPPORTED, bad
        for bad in (dict(k=A + 8), dict(v=A + 2), dict(kc=A + 4), dict(ks=A + 8), dict(vs=A + 1)):
            assert call(**bad) == b.FA_ERR_MISALIGNED, bad
        assert call(T=0, k=0, v=0, slots=0) == b.FA_OK
    for bad in (dict(kt=255), dict(kh=4), dict(vt=1), dict(vh=132)):
        assert store(**bad) == b.FA_ERR_MISALIGNED, bad


def test_attention_validation():
    own = dict(kc=A, ks=A, vc=A, vs=A, pages=4, page=16, H=2, d=128, kg=1.0, vg=1.0)
    ok = dict(q=A, qt=1024, qh=128, T=2, cu=A, max_q=1, table=A, width=4, lengths=A, B=2, heads=8, scale=0.1, o=A,
              ot=1024, oh=128, lse=A, ws=A, wsb=1 << 30)

    def call(**kw):
        a = {**ok, **kw}
        return b.fa_kv4_attn(cache({**own, **{n: x for n, x in kw.items() if n in own}}).address,
                             *(a[n] for n in ok), None)

    assert b.fa_kv4_attn(None, *ok.values(), None) == b.FA_ERR_INVALID_ARG

    for bad in (dict(T=-1), dict(B=-1), dict(max_q=-1), dict(heads=7), dict(H=0), dict(heads=-8), dict(pages=-1), dict(width=-1),
                dict(page=8), dict(scale=0.0), dict(scale=float("nan")), dict(kg=0.0), dict(vg=float("inf")),
                dict(q=0), dict(o=0), dict(lse=0), dict(lengths=0), dict(table=0), dict(kc=0), dict(width=1 << 28),
                dict(cu=0, T=1)):
        assert call(**bad) == b.FA_ERR_INVALID_ARG, bad
    for bad in (dict(d=80), dict(d=512)):
        assert call(**bad) == b.FA_ERR_UNSUPPORTED, bad
    for bad in (dict(q=A + 8), dict(o=A + 4), dict(vc=A + 2), dict(qt=1028), dict(qh=4), dict(ot=1), dict(oh=2)):
        assert call(**bad) == b.FA_ERR_MISALIGNED, bad
    # Few tokens need no workspace, many do.
    assert b.fa_kv4_attn_workspace_size(2, 8, 2, 128, 1, 16, 4) == 0
    need = b.fa_kv4_attn_workspace_size(2, 8, 2, 128, 1, 16, 1000)
    assert need > 0
    for bad in (dict(ws=0), dict(ws=A + 16), dict(wsb=need - 1)):
        assert call(width=1000, **bad) == b.FA_ERR_WORKSPACE, bad
    for empty in (dict(B=0), dict(T=0), dict(max_q=0)):
        assert call(**empty, q=0, o=0, lse=0, lengths=0, ws=0) == b.FA_OK
    for bad in ((-1, 8, 2, 128, 1, 16, 1000), (2, 7, 2, 128, 1, 16, 1000), (2, 8, 2, 100, 1, 16, 1000),
                (2, 8, 2, 128, -1, 16, 1000), (1 << 30, 8, 2, 128, 64, 16, 1000), (2, 8, 2, 128, 1, 17, 1000),
                (2, 8, 2, 128, 1, 16, 1 << 28)):
        assert b.fa_kv4_attn_workspace_size(*bad) == 0


def _cache():
    def u8(*s):
        return torch.zeros(s, dtype=torch.uint8)
    return u8(4, 2, 16, 64), u8(4, 2, 16, 8), u8(4, 2, 16, 64), u8(4, 2, 16, 8)


def test_torch_layer_refuses_host_tensors_and_wrong_kinds():
    i32 = torch.zeros(2, dtype=torch.int32)
    table = torch.zeros((2, 4), dtype=torch.int32)
    one = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="contiguous CUDA"):
        api.page_grow(i32, i32, table, i32, one, 16, 4)
    with pytest.raises(ValueError, match="page_size"):
        api.page_slots(i32, i32, table, 24, 4)
    with pytest.raises(ValueError, match="num_tokens"):
        api.page_slots(i32, i32, table, 16, -1)
    with pytest.raises(ValueError, match="not torch.int64"):
        api.page_slots(i32.long(), i32, table, 16, 4)
    with pytest.raises(ValueError, match="1-D"):
        api.page_slots(table, i32, table, 16, 4)
    with pytest.raises(ValueError, match="contiguous CUDA"):
        api.KV4Cache(*_cache())
    with pytest.raises(ValueError, match="shape"):
        api.KV4Cache(torch.zeros(4, dtype=torch.uint8), *_cache()[1:])
    with pytest.raises(ValueError, match="uint8"):
        api.KV4Cache(_cache()[0].int(), *_cache()[1:])
    with pytest.raises(TypeError):
        api.KV4Cache(None, *_cache()[1:])


def test_gains_whose_products_could_overflow_are_refused():
    for gain, want in ((2.0 ** -100, b.FA_OK), (2.0 ** 100, b.FA_OK), (2.0 ** -101, b.FA_ERR_INVALID_ARG),
                       (2.0 ** 100 * 1.001, b.FA_ERR_INVALID_ARG)):
        for own in (dict(kg=gain, vg=1.0), dict(kg=1.0, vg=gain)):
            desc = cache(dict(kc=A, ks=A, vc=A, vs=A, pages=3, page=16, H=2, d=128, **own))
            assert b.fa_kv4_store(desc.address, A, A, 256, 128, 256, 128, A, 0, None) == want
            assert b.fa_kv4_load(desc.address, A, 0, A, A, None) == want


def test_attention_of_row_counts_past_31_bits_is_refused():
    desc = cache(dict(kc=A, ks=A, vc=A, vs=A, pages=4, page=16, H=1, d=128, kg=1.0, vg=1.0))
    top = (1 << 31) - 1
    for batch, heads, max_q in ((2, 8, top), (top, top, top), (top, 64, 1)):
        args = [A, 1024, 128, 2, A, max_q, A, 4, A, batch, heads, 0.1, A, 1024, 128, A, A, 1 << 60]
        assert b.fa_kv4_attn(desc.address, *args, None) == b.FA_ERR_INVALID_ARG
        assert b.fa_kv4_attn_workspace_size(batch, heads, 1, 128, max_q, 16, 4) == 0


def test_rows_that_overlap_are_no_output():
    rows = serving._rows
    x = torch.zeros(4096, dtype=torch.bfloat16)
    def layout(*stride, shape=(3, 2, 64)):
        return rows(x.as_strided(shape, (*stride, 1)), "out", None, -1, written=True)
    assert layout(128, 64) == (128, 64) and layout(64, 192) == (64, 192) and layout(136, 64) == (136, 64)
    assert layout(8, 64, shape=(1, 2, 64)) == (0, 64) and layout(64, 3, shape=(3, 1, 64)) == (64, 0)
    for bad in ((64, 64), (64, 128), (120, 64), (0, 64), (128, 56)):
        with pytest.raises(ValueError, match="overlap"):
            layout(*bad)


C_CLIENT = r"""
#include <stdio.h>
#include <stddef.h>
#include "fa_paged.h"

int main(void) {
  int fails = 0;
  fa_kv4_cache cache = {NULL, NULL, NULL, NULL, 0, 16, 2, 128, 1.0f, 1.0f};
  if (fa_kv4_store(&cache, NULL, NULL, 0, 0, 0, 0, NULL, 0, NULL) != FA_OK) fails |= 1;
  if (fa_kv4_load(&cache, NULL, 0, NULL, NULL, NULL) != FA_OK) fails |= 2;
  cache.d = 80;
  if (fa_kv4_load(&cache, NULL, 0, NULL, NULL, NULL) != FA_ERR_UNSUPPORTED) fails |= 4;
  if (fa_page_grow(NULL, NULL, NULL, 0, 0, 16, NULL, 0, NULL, 0, NULL, NULL, NULL, NULL, NULL) != FA_OK) fails |= 8;
  if (fa_page_slots(NULL, NULL, NULL, 1, 0, 16, 0, NULL, NULL, NULL) != FA_ERR_INVALID_ARG) fails |= 16;
  if (fa_kv4_attn_workspace_size(1, 8, 2, 128, 1, 16, 100000) == 0) fails |= 32;
  cache.d = 128;
  if (fa_kv4_attn(&cache, NULL, 0, 0, 0, NULL, 1, NULL, 0, NULL, 0, 8, 1.0f, NULL, 0, 0, NULL, NULL, 0, NULL) != FA_OK)
    fails |= 64;
  printf("%d\n", fails);
  return fails != 0;
}
"""


def test_header_is_plain_c_and_a_c_program_links_the_library(tmp_path):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("gcc not available")
    src, exe = tmp_path / "client.c", tmp_path / "client"
    src.write_text(C_CLIENT)
    libdir = os.path.dirname(b.LIB_PATH)
    r = subprocess.run([gcc, "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic", f"-I{build.INCLUDE}", str(src), "-o",
                        str(exe), f"-L{libdir}", "-l:libfa_gb300.so", f"-Wl,-rpath,{libdir}"], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert out.returncode == 0 and out.stdout.strip() == "0", out.stdout + out.stderr


def test_reference_codes_and_scales():
    assert R.e4m3_value(0x7E) == 448 and R.e4m3_value(0x7F) == 480 and R.e4m3_value(1) == 2.0 ** -9
    assert R.e4m3_value(0xB8) == 1.0  # the sign bit is ignored
    x = np.zeros((1, 16))
    x[0, :8] = [6, -6, 0.25, 0.75, 1.25, -1.75, 2.5, 5.0]  # scale 1: the ties go to even
    codes, scales = R.encode(x, 1.0)
    got = R.decode(codes, scales, 1.0)[0, :8]
    assert list(got) == [6, -6, 0, 1, 1, -2, 2, 4]
    x = np.full((1, 16), 1e9)
    assert np.all(R.decode(*R.encode(x, 1.0), 1.0) == 6 * 448)  # saturates
    assert np.all(R.decode(*R.encode(np.full((1, 16), 1e-9), 1.0), 1.0) == 0)


def test_reference_attention_on_one_key_and_two():
    k = np.zeros((1, 1, 16, 64))
    v = np.zeros((1, 1, 16, 64))
    k[0, 0, 0, 0], k[0, 0, 1, 0] = 1.0, 3.0
    v[0, 0, 0, 0], v[0, 0, 1, 0] = 10.0, 20.0
    q = np.zeros((2, 1, 64))
    q[:, 0, 0] = 0.5
    o, lse, _, _, _ = R.attend(q, (k, v), np.zeros((1, 1), int), [2], [0, 2], 2, 1.0)
    w = 1 / (1 + math.exp(1.0))
    assert np.allclose(o[:, 0, 0], [10.0, 10 * w + 20 * (1 - w)]) and np.allclose(lse[:, 0], [0.5, math.log(math.exp(0.5) + math.exp(1.5))])


def test_reference_pages_by_hand():
    slots, cu, table, held, left = R.pages([15, 0, 32], [3, 1, 0], np.full((3, 2), 9), [5, 6, 7], 3, 16, 6)
    assert list(cu) == [0, 3, 4, 4] and list(held) == [18, 1, 32] and left == 1
    assert list(slots) == [9 * 16 + 15, 7 * 16, 7 * 16 + 1, 6 * 16, -1, -1]
    assert table.tolist() == [[9, 7], [6, 9], [9, 9]]


def test_numbers_past_31_bits_are_refused_not_cut():
    i32 = torch.zeros(2, dtype=torch.int32)
    table = torch.zeros((2, 4), dtype=torch.int32)
    for tokens in (1 << 31, (1 << 32) + 4):
        with pytest.raises(ValueError, match="2\\^31"):
            api.page_slots(i32, i32, table, 16, tokens)
        with pytest.raises(ValueError, match="2\\^31"):
            api.page_grow(i32, i32, table, i32, i32[:1], 16, tokens)
    for sizes in ((1 << 31, 8, 4, 1), (2, 1 << 32, 4, 1), (2, 8, (1 << 32) + 4, 1), (2, 8, 4, (1 << 32) + 1)):
        batch, heads, width, max_q = sizes
        with pytest.raises(ValueError, match="2\\^31"):
            api.kv4_attention_workspace_bytes(batch, heads, None, width, max_q)
    with pytest.raises(ValueError, match="2\\^31"):
        serving._slot_count(torch.empty((1 << 32) + 1, dtype=torch.int64, device="meta"), -1)


@pytest.mark.parametrize("head_dim", [65, 79, 129, 80, 0, 512])
def test_empty_cache_of_an_unsupported_head_dimension_is_refused(head_dim, monkeypatch):
    monkeypatch.setattr(serving, "_dense", lambda *a: None)  # (the arrays are on the host here)
    with pytest.raises(ValueError, match="head dimension"):
        api.KV4Cache.empty(2, 1, 16, head_dim, device="cpu")
    assert api.KV4Cache.empty(2, 1, 16, 64, device="cpu").head_dim == 64


def test_index_arrays_off_their_alignment_are_refused():
    """A kernel that read them would raise a misaligned-address fault."""
    grow = dict(lengths=A, new=A, table=A, B=2, width=4, page=16, free=A, free_size=9, count=A, T=8, slots=A, cu=A,
                held=A, out=A)
    for name in ("lengths", "new", "table", "free", "count", "slots", "cu", "held", "out"):
        for off in (1, 2) + ((4,) if name == "slots" else ()):
            a = {**grow, name: A + off}
            assert b.fa_page_grow(*a.values(), None) == b.FA_ERR_MISALIGNED, (name, off)
            if name in ("lengths", "new", "table", "slots", "cu"):
                assert b.fa_page_slots(*(a[n] for n in ("lengths", "new", "table", "B", "width", "page", "T", "slots", "cu")),
                                       None) == b.FA_ERR_MISALIGNED, (name, off)
    desc = cache(dict(kc=A, ks=A, vc=A, vs=A, pages=3, page=16, H=2, d=128, kg=1.0, vg=1.0)).address
    for off in (1, 4):
        assert b.fa_kv4_store(desc, A, A, 256, 128, 256, 128, A + off, 4, None) == b.FA_ERR_MISALIGNED
        assert b.fa_kv4_load(desc, A + off, 4, A, A, None) == b.FA_ERR_MISALIGNED
    attn = dict(q=A, qt=1024, qh=128, T=2, cu=A, max_q=1, table=A, width=4, lengths=A, B=2, heads=8, scale=0.1, o=A,
                ot=1024, oh=128, lse=A, ws=A, wsb=1 << 30)
    for name in ("cu", "table", "lengths", "lse"):
        for off in (1, 2, 3):
            assert b.fa_kv4_attn(desc, *{**attn, name: A + off}.values(), None) == b.FA_ERR_MISALIGNED, (name, off)


OLD_PROFILE = r"""
#include <stdio.h>
#include <string.h>
#include "fa_paged.h"

/* The record as it was before there were serving calls, and what lies behind it. */
struct { int launches[9]; double ms[9]; unsigned char behind[256]; } old;

int main(void) {
  int fails = 0, i, launches[20];
  double ms[20];
  memset(&old, 0xa5, sizeof(old));
  fa_profile_start();
  if (fa_profile_stop((fa_profile*)&old) != FA_OK) fails |= 1;
  for (i = 0; i < 9; ++i) if (old.launches[i] != 0 || old.ms[i] != 0) fails |= 2;
  for (i = 0; i < 256; ++i) if (old.behind[i] != 0xa5) fails |= 4;
  if (fa_profile_stop(NULL) != FA_OK || fa_profile_stop_kinds(5, NULL, NULL) != FA_OK) fails |= 8;
  if (fa_profile_stop_kinds(-1, launches, ms) != FA_ERR_INVALID_ARG) fails |= 16;
  memset(launches, 0xa5, sizeof(launches)), memset(ms, 0xa5, sizeof(ms));
  if (fa_profile_stop_kinds(FA_KERNEL_ALL_KINDS, launches, ms) != FA_OK) fails |= 32;
  for (i = 0; i < 20; ++i) if ((launches[i] == 0 && ms[i] == 0) != (i < FA_KERNEL_ALL_KINDS)) fails |= 64;
  if (strcmp(fa_kernel_name(FA_KERNEL_KINDS), "page") || strcmp(fa_kernel_name(FA_KERNEL_ALL_KINDS), "unknown")) fails |= 128;
  printf("%d\n", fails);
  return fails != 0;
}
"""


def test_a_profile_record_of_an_older_program_is_not_written_past(tmp_path):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("gcc not available")
    src, exe = tmp_path / "client.c", tmp_path / "client"
    src.write_text(OLD_PROFILE)
    libdir = os.path.dirname(b.LIB_PATH)
    r = subprocess.run([gcc, "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic", f"-I{build.INCLUDE}", str(src), "-o",
                        str(exe), f"-L{libdir}", "-l:libfa_gb300.so", f"-Wl,-rpath,{libdir}"], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert out.returncode == 0 and out.stdout.strip() == "0", out.stdout + out.stderr


def test_the_message_of_a_misaligned_argument_fits_index_arrays():
    text = b.fa_strerror(b.FA_ERR_MISALIGNED)
    assert "aligned" in text and "16" not in text
