"""Attention over packed sequences, norms and rotation, rotated append: argument checks (nothing
is launched), the layout of the argument structures, and the references' gradients."""

import os
import shutil
import subprocess

import pytest
import torch

import packed_ref as P
import rotary_ref as R
from tiled_attention_tmem_gb300 import api, build
from tiled_attention_tmem_gb300 import binding as b

A = 1 << 20  # an aligned fake address; never dereferenced


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build_library()
    return b.lib()


def rows(data=A, token=1024, head=128):
    return data, token, head


# ------------------------------------------------------------------ attention

SHAPE = dict(B=2, T=10, H=8, Hkv=2, d=128, scale=0.1, causal=1)
FWD_BAD = [
    (b.FA_ERR_INVALID_ARG, [dict(B=-1), dict(T=-1), dict(H=-8), dict(Hkv=-2), dict(H=7), dict(Hkv=0), dict(causal=2),
                            dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
                            dict(q=rows(0)), dict(k=rows(0)), dict(v=rows(0)), dict(lse=0), dict(cu=0),
                            dict(q=rows(token=0)), dict(k=rows(token=-1024)), dict(v=rows(head=0)),
                            dict(q=rows(token=1 << 34)), dict(T=(1 << 30) + 1), dict(T=1 << 29), dict(B=1 << 30)]),
    (b.FA_ERR_UNSUPPORTED, [dict(d=80), dict(d=512), dict(d=0), dict(H=66)]),
    (b.FA_ERR_MISALIGNED, [dict(q=rows(A + 8)), dict(k=rows(A + 2)), dict(q=rows(token=1028)), dict(v=rows(head=4)),
                           dict(lse=A + 2), dict(cu=A + 1)]),
    (b.FA_ERR_WORKSPACE, [dict(B=40, ws=0), dict(B=40, ws=A + 16), dict(B=40, short=1)]),
]


def call_fwd(q=rows(), k=rows(), v=rows(), o=rows(), lse=A, cu=A, ws=A, short=0, **kw):
    s = {**SHAPE, **kw}
    need = b.fa_packed_fwd_workspace_size(*(s[n] for n in ("B", "T", "H", "Hkv", "d")))
    return b.fa_packed_fwd(*q, *k, *v, *o, lse, cu, s["B"], s["T"], s["H"], s["Hkv"], s["d"], s["scale"], s["causal"], ws,
                           max(need - short, 0), 0)


def call_bwd(q=rows(), k=rows(), v=rows(), o=rows(), do=rows(), lse=A, dq=rows(), dk=rows(), dv=rows(), cu=A, ws=A,
             short=0, variant=0, **kw):
    s = {**SHAPE, **kw}
    need = b.fa_packed_bwd_workspace_size(*(s[n] for n in ("B", "T", "H", "Hkv", "d")), variant)
    return b.fa_packed_bwd(*q, *k, *v, *o, *do, lse, *dq, *dk, *dv, cu, s["B"], s["T"], s["H"], s["Hkv"], s["d"],
                           s["scale"], s["causal"], variant, ws, max(need - short, 0), 0)


@pytest.mark.parametrize("status,bad", FWD_BAD)
def test_attention_refuses(status, bad):
    for kw in bad:
        assert call_fwd(**kw) == status, kw
        assert call_bwd(**kw) == status, kw
    for kw in (dict(o=rows(0)),) if status == b.FA_ERR_INVALID_ARG else ():
        assert call_fwd(**kw) == status and call_bwd(**kw) == status
    more = {b.FA_ERR_INVALID_ARG: [dict(variant=3), dict(do=rows(0)), dict(dq=rows(0)), dict(dv=rows(0)), dict(dk=rows(token=0))],
            b.FA_ERR_UNSUPPORTED: [dict(variant=5, d=192), dict(variant=5, d=384)],
            b.FA_ERR_MISALIGNED: [dict(do=rows(A + 4)), dict(dk=rows(head=12))],
            b.FA_ERR_WORKSPACE: [dict(variant=7, short=1)]}[status]
    for kw in more:
        assert call_bwd(**kw) == status, kw


def test_attention_without_work_touches_nothing():
    none = dict(q=rows(0), k=rows(0), v=rows(0), o=rows(0), lse=0, cu=0, ws=0)
    for kw in (dict(T=0), dict(H=0, Hkv=0), dict(H=0)):
        assert call_fwd(**kw, **none) == b.FA_OK and call_bwd(**kw, **none, do=rows(0), dq=rows(0)) == b.FA_OK
    assert call_fwd(B=0, **none) == b.FA_OK
    assert b.lib().fa_packed_fwd(None) == b.FA_ERR_INVALID_ARG and b.lib().fa_packed_bwd(None) == b.FA_ERR_INVALID_ARG


def test_attention_workspace_sizes():
    # The forward needs none for few sequences and items; both bounds (32 sequences, two items an SM).
    assert b.fa_packed_fwd_workspace_size(3, 100, 8, 2, 128) == 0 == b.fa_packed_fwd_workspace_size(32, 100, 8, 2, 128)
    assert b.fa_packed_fwd_workspace_size(33, 100, 8, 2, 128) >= 33 * 16
    assert b.fa_packed_fwd_workspace_size(3, 100000, 8, 2, 128) >= 3 * 16
    five = b.fa_packed_bwd_workspace_size(3, 100, 8, 2, 128, 5)
    seven = b.fa_packed_bwd_workspace_size(3, 100, 8, 2, 128, 7)
    # The fp32 dQ of 100 tokens and what the sequences' last tiles round up; AUTO runs the 5-GEMM form.
    assert five - seven > 4 * 100 * 8 * 128 - 3 * 2 * 128 * 1 and b.fa_packed_bwd_workspace_size(3, 100, 8, 2, 128, 0) == five
    for bad in ((-1, 100, 8, 2, 128), (3, 100, 7, 2, 128), (3, 100, 8, 2, 100), (3, 100, 66, 2, 128), (3, 0, 8, 2, 128)):
        assert b.fa_packed_fwd_workspace_size(*bad) == 0 and b.fa_packed_bwd_workspace_size(*bad, 0) == 0
    assert b.fa_packed_bwd_workspace_size(3, 100, 8, 2, 256, 5) == 0


# ------------------------------------------------------------------ norms, rotation, append

def call_rope(q=rows(), k=rows(), qo=rows(), ko=rows(), rotary=A, pos=A, wq=A, wk=A, P=16, rot=64, eps=1e-6, inter=0, T=4,
              H=8, Hkv=2, d=128):
    return b.fa_qk_norm_rope(*q, *k, *qo, *ko, rotary, pos, wq, wk, P, rot, eps, inter, T, H, Hkv, d, 0)


def call_rope_bwd(gq=rows(), gk=rows(), q=rows(), k=rows(), qo=rows(), ko=rows(), rotary=A, pos=A, wq=A, wk=A, dwq=A, dwk=A,
                  P=16, rot=64, eps=1e-6, inter=0, T=4, H=8, Hkv=2, d=128, ws=A, short=0):
    need = b.fa_qk_norm_rope_bwd_workspace_size(T, H, Hkv, d)
    return b.fa_qk_norm_rope_bwd(*gq, *gk, *q, *k, *qo, *ko, rotary, pos, wq, wk, dwq, dwk, P, rot, eps, inter, T, H, Hkv, d,
                                 ws, max(need - short, 0), 0)


def cache(**kw):
    c = {**dict(kc=A, ks=A, vc=A, vs=A, pages=3, page=16, Hkv=2, d=128, kg=1.0, vg=1.0), **kw}
    return b.FaKv4Cache(c["kc"], c["ks"], c["vc"], c["vs"], c["pages"], c["page"], c["Hkv"], c["d"], c["kg"], c["vg"])


def call_append(q=rows(), k=rows(), v=rows(), qo=rows(), ko=rows(), rotary=A, pos=A, wq=A, wk=A, slots=A, P=16, rot=64,
                eps=1e-6, inter=0, T=4, H=8, **kw):
    desc = cache(**kw)
    return b.fa_kv4_append(desc.address, *q, *k, *v, *qo, *ko, rotary, pos, wq, wk, slots, P, rot, eps, inter, T, H, 0)


COMMON = [
    (b.FA_ERR_INVALID_ARG, [dict(T=-1), dict(H=-1), dict(P=-1), dict(rot=-32), dict(inter=2), dict(eps=-1.0),
                            dict(eps=float("nan")), dict(eps=float("inf")), dict(pos=0), dict(rotary=0), dict(q=rows(0)),
                            dict(qo=rows(0)), dict(k=rows(0)), dict(H=65536), dict(T=(1 << 30) + 1)]),
    (b.FA_ERR_UNSUPPORTED, [dict(d=80), dict(rot=160), dict(rot=16), dict(rot=48)]),
    (b.FA_ERR_MISALIGNED, [dict(q=rows(A + 8)), dict(k=rows(token=1028)), dict(qo=rows(head=4)), dict(rotary=A + 4),
                           dict(pos=A + 2), dict(wq=A + 2), dict(wk=A + 8)]),
]


@pytest.mark.parametrize("status,bad", COMMON)
def test_rotation_and_append_refuse(status, bad):
    for kw in bad:
        assert call_rope(**kw) == status, kw
        assert call_rope_bwd(**kw) == status, kw
        assert call_append(**kw) == status, kw
    if status == b.FA_ERR_INVALID_ARG:
        assert call_rope(ko=rows(0)) == status and call_rope(Hkv=-1) == status and call_rope(H=0, Hkv=40000) == status
        for kw in (dict(gq=rows(0)), dict(gk=rows(0)), dict(dwq=0), dict(dwk=0)):
            assert call_rope_bwd(**kw) == status, kw
        for kw in (dict(v=rows(0)), dict(slots=0), dict(page=24), dict(kg=0.0), dict(kc=0), dict(pages=-1)):
            assert call_append(**kw) == status, kw
    if status == b.FA_ERR_MISALIGNED:
        for kw in (dict(dwq=A + 2), dict(gk=rows(A + 4))):
            assert call_rope_bwd(**kw) == status, kw
        for kw in (dict(slots=A + 4), dict(v=rows(head=4)), dict(ko=rows(A + 2)), dict(ks=A + 8)):
            assert call_append(**kw) == status, kw
    for ws in (dict(ws=0), dict(ws=A + 16), dict(short=1)):
        assert call_rope_bwd(**ws) == b.FA_ERR_WORKSPACE


def test_rotation_without_work_touches_nothing():
    none = dict(q=rows(0), k=rows(0), qo=rows(0), ko=rows(0), rotary=0, pos=0, wq=0, wk=0)
    assert call_rope(T=0, **none) == b.FA_OK and call_rope(H=0, Hkv=0, **none) == b.FA_OK
    assert call_rope_bwd(T=0, **none, gq=rows(0), gk=rows(0), dwq=0, dwk=0, ws=0) == b.FA_OK
    assert call_append(T=0, **none, v=rows(0), slots=0) == b.FA_OK
    for f in ("fa_qk_norm_rope", "fa_qk_norm_rope_bwd", "fa_kv4_append"):
        assert getattr(b.lib(), f)(None) == b.FA_ERR_INVALID_ARG
    assert b.fa_qk_norm_rope_bwd_workspace_size(0, 8, 2, 128) == 0
    assert b.fa_qk_norm_rope_bwd_workspace_size(5, 8, 2, 100) == 0


# ------------------------------------------------------------------ the torch layer

def test_torch_layer_refuses_host_tensors_and_wrong_kinds():
    bf, i32 = torch.bfloat16, torch.int32
    x = torch.zeros((4, 2, 64), dtype=bf)
    cu = torch.zeros(2, dtype=i32)
    for f in (lambda: api.packed_attention_forward(x, x, x, cu),
              lambda: api.packed_attention_backward(x, x, x, x, x, torch.zeros(4, 2), cu),
              lambda: api.qk_norm_rope(x, x, torch.zeros(8, 64), torch.zeros(4, dtype=i32)),
              lambda: api.qk_norm_rope_backward(x, x, x, x, torch.zeros(8, 64), torch.zeros(4, dtype=i32))):
        with pytest.raises(ValueError, match="CUDA bfloat16"):
            f()
    with pytest.raises(TypeError):
        api.packed_attention_forward(None, x, x, cu)
    with pytest.raises(ValueError, match="sizes"):
        api.packed_forward_workspace_bytes(1 << 31, 4, 2, 2, 64)
    with pytest.raises(ValueError, match="sizes"):
        api.packed_backward_workspace_bytes(1, 1 << 31, 2, 2, 64)
    import tiled_attention_tmem_gb300 as pkg
    assert pkg.packed_attention_forward is api.packed_attention_forward and pkg.kv4_append is api.kv4_append


# ------------------------------------------------------------------ the header

C_CLIENT = r"""
#include <stdio.h>
#include <stddef.h>
#include "fa_packed.h"

int main(void) {
  fa_packed_fwd_args f = {0};
  fa_qk_norm_rope_args r = {0};
  int fails = 0;
  f.H = 8, f.Hkv = 2, f.d = 128, f.scale = 0.1f, f.causal = 1;
  if (fa_packed_fwd(&f) != FA_OK) fails |= 1;
  f.d = 80;
  if (fa_packed_fwd(&f) != FA_ERR_UNSUPPORTED) fails |= 2;
  r.H = 8, r.Hkv = 2, r.d = 128;
  if (fa_qk_norm_rope(&r) != FA_OK) fails |= 4;
  if (fa_packed_fwd_workspace_size(40, 10, 8, 2, 128) == 0) fails |= 8;
  printf("%d %d %d %d %d %d\n", fails, (int)sizeof(fa_packed_fwd_args), (int)sizeof(fa_packed_bwd_args),
         (int)sizeof(fa_qk_norm_rope_args), (int)sizeof(fa_qk_norm_rope_bwd_args), (int)sizeof(fa_kv4_append_args));
  printf("%d %d %d %d %d %d\n", (int)offsetof(fa_packed_fwd_args, stream), (int)offsetof(fa_packed_bwd_args, variant),
         (int)offsetof(fa_qk_norm_rope_args, eps), (int)offsetof(fa_qk_norm_rope_bwd_args, workspace_bytes),
         (int)offsetof(fa_kv4_append_args, slots), (int)offsetof(fa_packed_bwd_args, cu));
  return fails != 0;
}
"""


def test_header_is_plain_c_and_its_structures_are_what_the_binding_packs(tmp_path):
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
    assert out.returncode == 0, out.stdout + out.stderr
    sizes, offsets = ([int(x) for x in line.split()] for line in out.stdout.strip().splitlines())
    forms = (b._PACKED_FWD, b._PACKED_BWD, b._QK_NORM_ROPE, b._QK_NORM_ROPE_BWD, b._KV4_APPEND)
    assert sizes == [0] + [f.size for f in forms]

    def at(form, field):  # where the field-th value is packed
        count = len(form.unpack(bytes(form.size)))
        values = [0] * count
        values[field] = 1
        return form.pack(*values).index(b"\x01") if form.pack(*values).count(b"\x01") else None

    assert offsets[0] == at(b._PACKED_FWD, 23) and offsets[4] == at(b._KV4_APPEND, 20)
    assert offsets[1] == at(b._PACKED_BWD, 33) and offsets[5] == at(b._PACKED_BWD, 25)
    assert offsets[3] == at(b._QK_NORM_ROPE_BWD, 33)


# ------------------------------------------------------------------ waits

WAITS = r"""
#include <stdio.h>
#include "ragged.cuh"
int main() {
  for (long long n = 0; n <= 1LL << 28; n = n ? 4 * n : 1) printf("%lld %lld\n", n, fa::ragged_wait_limit((int)n));
  return 0;
}
"""


def test_the_scheduling_warp_waits_for_the_longest_item(tmp_path):
    """An item of the dK/dV kernel takes a step for each query tile of its sequence; with 32 heads to a kv head a tile
    of 32 or 64 rows is 1 or 2 tokens.  A step is 2200 cycles; twice that is to be waited for, beyond the
    two seconds that every wait has, up to the longest sequence that is taken."""
    src, exe = tmp_path / "waits.cu", tmp_path / "waits"
    src.write_text(WAITS)
    r = subprocess.run([build.nvcc(), *build.ARCH, "-std=c++17", f"-I{build.CSRC}", f"-I{build.INCLUDE}", str(src), "-o", str(exe)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    limits = {int(n): int(x) for n, x in (line.split() for line in out.stdout.splitlines())}
    assert max(limits) == 1 << 28 and limits[0] >= 4e9
    assert all(x >= 4e9 + 2 * 2200 * n for n, x in limits.items())


# ------------------------------------------------------------------ the references

def test_reference_attention_gradients_are_those_of_differences():
    g = torch.Generator().manual_seed(1)
    q, k, v, do = (torch.randn((7, h, 4), generator=g, dtype=torch.float64) for h in (4, 2, 2, 4))
    cu = [0, 3, 3, 7]
    for causal in (True, False):
        r = P.attend(q, k, v, cu, 0.7, causal, do)
        for name, t in (("dq", q), ("dk", k), ("dv", v)):
            for at in ((0, 0, 1), (2, 1, 3), (5, 1, 0), (6, 0, 2)):
                if at[1] >= t.shape[1]:
                    continue
                h, both = 1e-6, []
                for sign in (1, -1):
                    t[at] += sign * h
                    both.append(float((P.attend(q, k, v, cu, 0.7, causal)["o"] * do).sum()))
                    t[at] -= sign * h
                # Central differences of h = 1e-6: h^2 of the third derivative and 2^-52 / h.
                assert abs((both[0] - both[1]) / (2 * h) - float(r[name][at])) < 1e-7


def test_reference_attention_keeps_sequences_apart():
    g = torch.Generator().manual_seed(2)
    q, k, v = (torch.randn((9, 2, 8), generator=g, dtype=torch.float64) for _ in range(3))
    r = P.attend(q, k, v, [1, 4, 9], 0.3, True)
    assert bool(torch.isnan(r["lse"][0]).all()) and bool(torch.isfinite(r["lse"][1:]).all())
    assert torch.equal(r["o"][1], v[1]) and torch.equal(r["o"][4], v[4])  # first tokens see themselves


@pytest.mark.parametrize("interleaved", (False, True))
@pytest.mark.parametrize("weight", (True, False))
def test_reference_rotation_gradients_are_those_of_differences(weight, interleaved):
    g = torch.Generator().manual_seed(3)
    x, dy = (torch.randn((5, 2, 12), generator=g, dtype=torch.float64) for _ in range(2))
    w = torch.randn(12, generator=g, dtype=torch.float64) if weight else None
    rotary, pos = R.table(6, 8), torch.tensor([0, 5, -1, 3, 6])
    mine = R.live(pos, rotary)

    def value():
        return float((R.forward(x, w, 1e-3, rotary, pos, interleaved)[0] * dy)[mine].sum())

    dx, _, dw, _ = R.backward(dy, x, w, 1e-3, rotary, pos, interleaved)
    for t, grad, places in ((x, dx, ((0, 0, 0), (1, 1, 7), (2, 0, 3), (3, 1, 11), (4, 0, 0))), (w, dw, (0, 5, 11))):
        for at in places if t is not None else ():
            h, both = 1e-6, []
            for sign in (1, -1):
                t[at] += sign * h
                both.append(value())
                t[at] -= sign * h
            assert abs((both[0] - both[1]) / (2 * h) - float(grad[at])) < 1e-7
    # A rotation keeps lengths, and turns back.
    y = R.turn(x, rotary, pos.clamp(0, 5), interleaved)[0]
    assert torch.allclose(y.norm(dim=-1), x.norm(dim=-1), rtol=1e-6)
    assert torch.allclose(R.turn(y, rotary, pos.clamp(0, 5), interleaved, back=True)[0], x, atol=1e-6)
