"""The steps on drafted tokens on the host: struct layout, workspace sizes and refusals, all
before any launch (fake device pointers are never touched)."""
import ctypes
import os
import subprocess
import tempfile

import pytest

from gated_delta_rule_depthwise_amd import binding as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
F = 1 << 20


def tape(**kw):
    a = dict(k=F, d=F, g=F, raw=None, len=F, cap=16)
    a.update(kw)
    return B.tape(a["k"], a["d"], a["g"], a["raw"], a["len"], a["cap"])


def draft(p, t=None, q=F, g=F, h=F, cs=None, cw=None, o=F, n=4, T=4, share=1, fn=B.gdn_draft):
    return fn(p, q, F, F, g, F, h, cs, cw, t or tape(), o, n, T, share, None)


def fold(p, t=None, h=F, cs=None, ho=2 * F, co=None, n=4, share=1, min_len=0, fn=B.gdn_fold):
    return fn(p, h, cs, ho, co, t or tape(), None, n, share, min_len, None)


def test_tape_struct_layout():
    fields = [f[0] for f in B.gdn_tape._fields_]
    prog = "#include <stddef.h>\n#include <stdio.h>\n#include \"gdn.h\"\nint main(void) {\n"
    prog += '  printf("%zu %d %d\\n", sizeof(gdn_tape), GDN_BAD_TAPE, GDN_DRAFT_MAX_T);\n'
    prog += "".join('  printf("%%zu\\n", offsetof(gdn_tape, %s));\n' % f for f in fields) + "  return 0;\n}\n"
    with tempfile.TemporaryDirectory() as d:
        src, exe = os.path.join(d, "l.c"), os.path.join(d, "l")
        open(src, "w").write(prog)
        subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), src, "-o", exe], check=True)
        out = [int(x) for x in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    assert out[:3] == [ctypes.sizeof(B.gdn_tape), B.GDN_BAD_TAPE, B.GDN_DRAFT_MAX_T]
    assert out[3:] == [getattr(B.gdn_tape, f).offset for f in fields]


@pytest.mark.parametrize("fn", [B.gdn_draft, B.kda_draft])
def test_draft_refusals(fn):
    p = B.params(2, 64, 64)

    def refused(status=B.GDN_E_ARG, params=p, **kw):
        assert draft(params, fn=fn, **kw) == status, kw

    for kw in (dict(T=0), dict(T=17), dict(T=-1), dict(n=0), dict(n=-4), dict(share=0), dict(share=3),
               dict(share=8), dict(q=None), dict(g=None), dict(h=None), dict(o=None), dict(o=F + 4),
               dict(q=F + 2), dict(t=tape(cap=0)), dict(t=tape(cap=3)), dict(t=tape(k=None)),
               dict(t=tape(d=None)), dict(t=tape(g=None)), dict(t=tape(len=None)), dict(t=tape(k=F + 4)),
               dict(t=tape(d=F + 8)), dict(t=tape(raw=F)), dict(cs=F), dict(cw=F),
               dict(n=1 << 30, T=16), dict(n=(1 << 21) + 1)):
        refused(**kw)
    if fn is B.kda_draft:
        refused(g=F + 4)
        refused(t=tape(g=F + 4))
    front = B.params(2, 64, 64, conv_k=4)
    refused(params=front, t=tape(raw=F), cs=F)                   # no taps
    refused(params=front, t=tape(raw=F), cw=F)                   # no windows
    refused(params=front, cs=F, cw=F)                            # no raw rows on the tape
    refused(params=front, t=tape(raw=F + 4), cs=F, cw=F)
    for bad in (B.params(2, 96, 96), B.params(2, 64, 128), B.params(2, 64, 64, dtype=7),
                B.params(2, 128, 128, dtype=B.GDN_F32), B.params(2, 64, 64, conv_k=5)):
        refused(B.GDN_E_UNSUPPORTED, params=bad)
    refused(params=B.params(2, 64, 64, ld_qkv=100))
    refused(params=B.params(4, 64, 64, Hqk=3))
    refused(params=B.params(2, 64, 64, z=F, norm_w=None))
    refused(params=B.params(2, 64, 64, z=F + 4, norm_w=F))
    assert fn(p, F, F, F, F, F, F, None, None, B.gdn_tape(), F, 4, 4, 1, None) == B.GDN_E_ARG
    lib = B.load()
    raw = lib.gdn_draft if fn is B.gdn_draft else lib.kda_draft
    assert raw(None, F, F, F, F, F, F, None, None, ctypes.byref(tape()), F, 4, 4, 1, None) == B.GDN_E_ARG
    assert raw(ctypes.byref(p), F, F, F, F, F, F, None, None, None, F, 4, 4, 1, None) == B.GDN_E_ARG


@pytest.mark.parametrize("fn", [B.gdn_fold, B.kda_fold])
def test_fold_refusals(fn):
    p, front = B.params(2, 64, 64), B.params(2, 64, 64, conv_k=3)
    for kw in (dict(n=0), dict(share=3), dict(share=0), dict(min_len=-1), dict(h=None), dict(ho=None),
               dict(t=tape(cap=0)), dict(t=tape(len=None)), dict(t=tape(raw=F)), dict(cs=F), dict(co=F),
               dict(share=2, ho=F)):                             # shared states are not written in place
        assert fold(p, fn=fn, **kw) == B.GDN_E_ARG, kw
    for kw in (dict(), dict(cs=F), dict(co=F), dict(cs=F, co=F), dict(cs=F, t=tape(raw=F))):
        assert fold(front, fn=fn, **kw) == B.GDN_E_ARG, kw
    assert fold(front, fn=fn, cs=F, co=F, t=tape(raw=F), share=2) == B.GDN_E_ARG   # nor shared windows
    assert fold(B.params(2, 64, 128), fn=fn) == B.GDN_E_UNSUPPORTED


def test_verify_workspace_and_refusals():
    assert B.gdn_verify_workspace_bytes(0, 1, 10) == 0
    assert B.gdn_verify_workspace_bytes((1 << 18) + 1, 1, 10) == 0
    assert B.gdn_verify_workspace_bytes(1, -1, 10) == 0
    assert B.gdn_verify_workspace_bytes(1, 1025, 10) == 0
    assert B.gdn_verify_workspace_bytes(1, 1, 0) == 0
    assert B.gdn_verify_workspace_bytes(1, 1, (1 << 30) + 1) == 0
    for V in (1, 4096, 4097, 50257, 262144, 262145, 1 << 30):
        n = B.gdn_verify_workspace_bytes(3, 2, V)
        assert 0 < n <= (3 * 64 * 16 + 255) // 256 * 256 and n % 256 == 0

    def call(target=F, ldt=100, q=F, ldq=100, dtype=B.GDN_F32, tok=F, u=F, n=2, T=3, V=100, acc=F, nxt=F,
             ws=F, nb=1 << 20):
        return B.gdn_verify(target, ldt, q, ldq, dtype, tok, None, u, n, T, V, acc, nxt, None, ws, nb, None)

    for kw in (dict(target=None), dict(u=None), dict(tok=None), dict(acc=None), dict(nxt=None), dict(ldt=99),
               dict(ldq=99), dict(n=0), dict(T=-1), dict(T=1025), dict(V=0), dict(target=F + 2),
               dict(q=F + 1), dict(dtype=B.GDN_BF16, target=F + 1), dict(ws=F + 8)):
        assert call(**kw) == B.GDN_E_ARG, kw
    assert call(dtype=2) == B.GDN_E_UNSUPPORTED
    assert call(nb=8) == B.GDN_E_WORKSPACE
    assert call(ws=None) == B.GDN_E_WORKSPACE
