"""The norm, rotary and tree-attention entry points without a GPU: their
structures' layouts against the header, the workspace query, and the refusals
that come before any launch."""
import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 20  # an aligned address that no refused call reads


def test_structures_match_the_header(w12lib, tmp_path):
    src = tmp_path / "sizes.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "w12.h"\nint main(void) {\n'
                   'printf("%zu %zu %zu", sizeof(w12_kv_cache), sizeof(w12_rope_args), sizeof(w12_attn_args));\n'
                   'printf(" %zu %zu %zu", offsetof(w12_rope_args, eps), offsetof(w12_attn_args, scale),\n'
                   '       offsetof(w12_kv_cache, page_stride));\nreturn 0;\n}\n')
    exe = tmp_path / "sizes"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), "-o", str(exe), str(src)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    assert got[:3] == [ctypes.sizeof(w12lib._Cache), w12lib._rope_args.size, w12lib._attn_args.size]
    rope = [0] * 23 + [1.0, 0, 0]  # eps is the 24th field
    assert w12lib._rope_args.pack(*rope)[got[3]:got[3] + 4] == b"\0\0\x80\x3f"
    attn = [0] * 17 + [1.0, 0.0, 0, 0, 0]
    assert w12lib._attn_args.pack(*attn)[got[4]:got[4] + 4] == b"\0\0\x80\x3f"
    assert w12lib._Cache.page_stride.offset == got[5]


def test_norm_refusals(w12lib):
    f = w12lib.load().w12_rmsnorm
    # x, ldx, residual, ldr, weight, eps, M, K, h_out, ldh, y, ldy, q8, ldq, scale, lds, stream
    base = dict(x=P, ldx=64, r=None, ldr=0, w=P, eps=1e-6, M=2, K=64, h=None, ldh=0, y=P, ldy=64, q=None, ldq=0, s=None,
                lds=0, st=None)

    def call(**change):
        return f(*{**base, **change}.values())

    assert call(M=0) == w12lib.W12_OK
    assert call(y=None) == w12lib.W12_OK  # no output asked for
    for change in (dict(M=-1), dict(K=0), dict(K=65537, ldx=65537, ldy=65537), dict(eps=-1.0), dict(eps=float("nan")),
                   dict(x=None), dict(w=None), dict(ldx=63), dict(ldy=63), dict(r=P, ldr=63), dict(h=P, ldh=63),
                   dict(q=P, ldq=64), dict(s=P, lds=1), dict(q=P, ldq=63, s=P, lds=1), dict(q=P, ldq=64, s=P, lds=0)):
        assert call(**change) == w12lib.W12_ERR_INVALID, change
    for change in (dict(x=P + 1), dict(w=P + 1), dict(y=P + 1), dict(r=P + 1, ldr=64), dict(h=P + 1, ldh=64),
                   dict(q=P, ldq=64, s=P + 2, lds=1)):
        assert call(**change) == w12lib.W12_ERR_ALIGN, change


def cache(w12lib, **change):
    c = w12lib._Cache(P, P, 4, 16, 2, 64, 2048, 128, 64)
    for name, value in change.items():
        setattr(c, name, value)
    return c


BAD_CACHES = [("W12_ERR_INVALID", dict(pages=-1)), ("W12_ERR_INVALID", dict(pages=2 ** 31)),
              ("W12_ERR_INVALID", dict(page_tokens=0)), ("W12_ERR_INVALID", dict(k=None)),
              ("W12_ERR_INVALID", dict(heads=0)), ("W12_ERR_INVALID", dict(token_stride=-128)),
              ("W12_ERR_ALIGN", dict(v=P + 8)), ("W12_ERR_ALIGN", dict(head_stride=60))]


def test_rope_refusals(w12lib):
    f = w12lib.load().w12_rope_append
    axis = ctypes.create_string_buffer(bytes([0] * 31 + [1]), 32)
    base = dict(q=P, k=P, v=P, ldq=256, ldk=128, ldv=128, qo=P, ko=P, ldqo=256, ldko=128, n=2, Hq=4, Hkv=2, dim=64, rot=64,
                inter=0, pos=P, ld_pos=2, axes=1, axis=0, freq=P, qn=0, kn=0, eps=1e-6, cache=0, slots=0)

    def call(c=None, **change):
        if c is not None:
            change["cache"], change["slots"] = ctypes.addressof(c), P
        return f(w12lib._rope_args.pack(*{**base, **change}.values()), None)

    assert f(None, None) == w12lib.W12_ERR_INVALID
    assert call(n=0) == w12lib.W12_OK
    for change in (dict(n=-1), dict(dim=32), dict(rot=8), dict(rot=80), dict(rot=-16), dict(inter=2), dict(eps=-1.0),
                   dict(Hq=0), dict(Hkv=0), dict(axes=0), dict(axes=5), dict(freq=0), dict(pos=0),
                   dict(axis=ctypes.addressof(axis)), dict(axes=2, ld_pos=1), dict(qo=0), dict(ko=0), dict(q=0),
                   dict(k=0), dict(q=0, qo=0, k=0, ko=0), dict(ldq=255), dict(ldqo=248), dict(ldk=120), dict(ldko=120),
                   dict(c=cache(w12lib), v=0), dict(c=cache(w12lib), ldv=120), dict(c=cache(w12lib, heads=3)),
                   dict(c=cache(w12lib, dim=128)), dict(slots=P)):
        assert call(**change) == w12lib.W12_ERR_INVALID, change
    for change in (dict(q=P + 8), dict(k=P + 8), dict(qo=P + 8), dict(ko=P + 2), dict(qn=P + 8), dict(pos=P + 2),
                   dict(ldq=260), dict(ldk=132), dict(c=cache(w12lib), v=P + 8), dict(c=cache(w12lib), ldv=132)):
        assert call(**change) == w12lib.W12_ERR_ALIGN, change
    for status, change in BAD_CACHES:
        assert call(c=cache(w12lib, **change)) == getattr(w12lib, status), change


def test_attn_workspace_query(w12lib):
    size = w12lib.load().w12_tree_attn_workspace_bytes
    assert 0 < size(0, 1, 1, 1, 64) <= size(1, 1, 40, 8, 128) < size(256, 8, 40, 8, 128) <= size(65536, 4096, 40, 8, 128)
    for bad in ((-1, 1, 8, 8, 64), (65537, 1, 8, 8, 64), (1, 0, 8, 8, 64), (1, 4097, 8, 8, 64), (1, 1, 9, 8, 64),
                (1, 1, 0, 8, 64), (1, 1, 8, 0, 64), (1, 1, 2048, 2048, 64), (1, 1, 8, 8, 96), (1, 1, 8, 8, 256)):
        assert size(*bad) == 0, bad


def test_attn_refusals(w12lib):
    lib = w12lib.load()
    base = dict(q=P, k=P, v=P, ldq=256, ldk=128, ldv=128, o=P, ldo=256, n=3, R=2, Hq=4, table=P, ld_table=4, width=4,
                ctx=P, parent=0, req=0, scale=0.0, cap=0.0, window=0, ctas=0, flags=0)
    need = lib.w12_tree_attn_workspace_bytes(3, 2, 4, 2, 64)

    def call(c=None, ws=P, nbytes=need, **change):
        args = w12lib._attn_args.pack(*{**base, **change}.values())
        return lib.w12_tree_attn(args, ctypes.addressof(c or cache(w12lib)), ws, nbytes, None)

    assert lib.w12_tree_attn(None, ctypes.addressof(cache(w12lib)), P, need, None) == w12lib.W12_ERR_INVALID
    assert call(n=0) == w12lib.W12_OK
    for change in (dict(n=-1), dict(n=65537), dict(R=0), dict(R=4097), dict(Hq=3), dict(width=-1), dict(ld_table=3),
                   dict(width=2 ** 27, ld_table=2 ** 27), dict(scale=-1.0), dict(cap=-1.0), dict(cap=1025.0),
                   dict(cap=float("inf")), dict(window=-1), dict(ctas=-1), dict(flags=2), dict(q=0), dict(k=0), dict(v=0),
                   dict(o=0), dict(ctx=0), dict(table=0), dict(ldq=248), dict(ldk=120), dict(ldv=120), dict(ldo=248)):
        assert call(**change) == w12lib.W12_ERR_INVALID, change
    for change in (dict(q=P + 8), dict(k=P + 8), dict(v=P + 8), dict(o=P + 8), dict(ldq=260), dict(ldo=260), dict(ws=P + 8),
                   dict(table=P + 2), dict(ctx=P + 2), dict(parent=P + 2), dict(req=P + 1)):
        assert call(**change) == w12lib.W12_ERR_ALIGN, change
    assert call(ws=None) == call(nbytes=need - 1) == w12lib.W12_ERR_CAPACITY
    for status, change in BAD_CACHES:
        assert call(c=cache(w12lib, **change)) == getattr(w12lib, status), change
    assert lib.w12_tree_attn_status(None, 256, None) == w12lib.W12_ERR_INVALID
    assert lib.w12_tree_attn_status(P, 255, None) == w12lib.W12_ERR_INVALID
