"""The norm and rotary entry points without a GPU: sizes, strides and options are checked on the
host before any launch."""
import ctypes

import pytest
import torch

from exact_attention_126_b200 import build, fa

A = 0x10000  # a fake, aligned device address: never dereferenced on these paths


@pytest.fixture(scope="module")
def lib():
    build.build()
    return fa.library()


def rows(data=A, heads=2, d=64, N=5, packed=False, **kw):
    st = dict(batch_stride=0 if packed else N * heads * d, token_stride=heads * d, head_stride=d)
    st.update(kw)
    return fa.fa_heads_t(data, heads, st["batch_stride"], st["token_stride"], st["head_stride"])


def params(**kw):
    p = dict(eps=1e-6, norm=1, rotary_dim=64, axes=1, inv_freq=A)
    p.update(kw)
    return fa.fa_norm_rope_t(**p)


def fwd(lib, q=None, k=None, v=None, qo=None, ko=None, vo=None, B=2, N=5, d=64, p=None):
    q, k = q or rows(), k or rows()
    return lib.fa_qk_norm_rope_fwd(q, k, v, qo or rows(heads=q.heads), ko or rows(heads=k.heads),
                                   vo, B, N, d, p or params(), None)


def test_forward_refusals(lib):
    assert fwd(lib, d=96) == 2
    assert fwd(lib, B=-1) == 1
    assert fwd(lib, N=-1) == 1
    assert fwd(lib, q=rows(data=A + 8)) == 3
    assert fwd(lib, q=rows(data=None)) == 1
    assert fwd(lib, q=rows(heads=-1)) == 1
    assert fwd(lib, q=rows(head_stride=60)) == 3
    assert fwd(lib, q=rows(token_stride=-128)) == 1
    assert fwd(lib, q=rows(batch_stride=1 << 41)) == 1
    assert fwd(lib, ko=rows(heads=3)) == 1              # both sides have the same heads
    assert fwd(lib, v=rows()) == 1                      # values need a place to go
    assert fwd(lib, vo=rows()) == 1
    assert fwd(lib, qo=rows(token_stride=0)) == 1       # written rows must not overlap
    assert fwd(lib, qo=rows(head_stride=32)) == 1
    assert fwd(lib, qo=rows(batch_stride=64)) == 1
    assert fwd(lib, B=1 << 20, N=1 << 10) == 2          # 2^31 elements and more
    assert fwd(lib, B=1 << 16, N=1 << 15) == 2
    assert fwd(lib, q=rows(batch_stride=1 << 34)) == 2  # rows further apart than 2^34 elements
    assert lib.fa_qk_norm_rope_fwd(rows(), rows(), None, rows(), rows(), None, 2, 5, 64, None,
                                   None) == 1


def test_parameter_refusals(lib):
    assert fwd(lib, p=params(rotary_dim=-16)) == 1
    assert fwd(lib, p=params(rotary_dim=20)) == 2
    assert fwd(lib, p=params(rotary_dim=80)) == 2
    assert fwd(lib, p=params(inv_freq=None)) == 1
    assert fwd(lib, p=params(inv_freq=A + 2)) == 3
    assert fwd(lib, p=params(axes=0)) == 1
    assert fwd(lib, p=params(axes=4, positions=A, pair_axis=A)) == 2
    assert fwd(lib, p=params(axes=2, pair_axis=A)) == 1  # several axes need positions
    assert fwd(lib, p=params(axes=2, positions=A)) == 1  # and an axis for each rotation
    assert fwd(lib, p=params(positions=A + 2)) == 3
    assert fwd(lib, p=params(eps=-1.0)) == 1
    assert fwd(lib, p=params(eps=float("nan"))) == 1
    assert fwd(lib, p=params(norm=0, q_weight=A)) == 1
    assert fwd(lib, p=params(q_weight=A + 1)) == 3
    assert fwd(lib, p=params(seq_lengths=A + 2)) == 3
    assert fwd(lib, p=params(cu_seqlens=A, seq_lengths=A, total_tokens=5)) == 1
    assert fwd(lib, p=params(cu_seqlens=A, total_tokens=-5)) == 1
    assert fwd(lib, p=params(cu_seqlens=A + 2, total_tokens=5)) == 3


def test_empty_calls(lib):
    none = rows(data=None, heads=0)
    assert fwd(lib, B=0, q=rows(data=None)) == 0
    assert fwd(lib, N=0, q=rows(data=None)) == 0
    assert fwd(lib, q=rows(data=None), p=params(cu_seqlens=A, total_tokens=0)) == 0
    assert fwd(lib, q=none, k=none, qo=none, ko=none) == 0


def test_backward_refusals(lib):
    assert lib.fa_qk_norm_rope_workspace_bytes(96) == 0
    need = lib.fa_qk_norm_rope_workspace_bytes(64)
    assert need > 0 and lib.fa_qk_norm_rope_workspace_bytes(128) == 2 * need

    def bwd(dq=None, q=rows(), k=rows(), gq=None, gqw=None, gkw=None, ws=A, n=need, p=None,
            d=64):
        return lib.fa_qk_norm_rope_bwd(dq or rows(), rows(), None, q, k, gq or rows(), rows(),
                                       None, gqw, gkw, 2, 5, d, p or params(), ws, n, None)

    assert bwd(q=None) == 1                     # the norm's gradient needs the inputs
    assert bwd(q=rows(heads=3)) == 1
    assert bwd(gq=rows(heads=3)) == 1
    assert bwd(gq=rows(token_stride=0)) == 1
    assert bwd(dq=rows(data=A + 2)) == 3
    assert bwd(gqw=A, p=params(norm=0)) == 1
    assert bwd(gqw=A + 2) == 3
    assert bwd(gqw=A, ws=None) == 1
    assert bwd(gkw=A, ws=A + 8) == 3
    assert bwd(gkw=A, n=need - 1) == 4
    assert bwd(d=32) == 2


def test_written_rows_that_others_use(lib):
    """Rows written at the data pointer of another kind, or of their own kind at other strides."""
    r = [rows(data=A * (i + 1)) for i in range(6)]
    p = ctypes.byref(params())
    fwd = lambda *t: lib.fa_qk_norm_rope_fwd(*t, 2, 5, 64, p, None)  # noqa
    assert fwd(r[0], r[1], r[2], r[3], r[3], r[5]) == 1
    assert fwd(r[0], r[1], r[2], r[1], r[4], r[5]) == 1
    assert fwd(r[0], r[1], r[2], r[3], r[4], r[0]) == 1
    head_major = rows(data=A, token_stride=64, head_stride=5 * 64)
    assert fwd(r[0], r[1], r[2], head_major, r[4], r[5]) == 1
    bwd = lambda *t: lib.fa_qk_norm_rope_bwd(*t, None, None, 2, 5, 64, p, None, 0, None)  # noqa
    g = [rows(data=A * (i + 7)) for i in range(3)]
    assert bwd(r[0], r[1], r[2], r[3], r[4], g[0], g[0], g[2]) == 1
    assert bwd(r[0], r[1], r[2], r[3], r[4], r[1], g[1], g[2]) == 1
    assert bwd(r[0], r[1], r[2], r[3], r[4], g[0], g[1], r[3]) == 1
    assert bwd(r[0], r[1], r[2], r[3], r[4], head_major, g[1], g[2]) == 1


def test_packed_single_tokens_in_place_at_other_strides(lib):
    """Sequences of one token each: the call steps through all of them by the token stride."""
    p = ctypes.byref(params(cu_seqlens=A, total_tokens=5))
    r = [rows(data=A * (i + 1)) for i in range(6)]
    wide = rows(data=A, token_stride=2 * r[0].token_stride)
    fwd = lambda *t: lib.fa_qk_norm_rope_fwd(*t, 5, 1, 64, p, None)  # noqa
    assert fwd(r[0], r[1], r[2], wide, r[4], r[5]) == 1
    assert fwd(wide, r[1], r[2], r[0], r[4], r[5]) == 1
    bwd = lambda *t: lib.fa_qk_norm_rope_bwd(*t, None, None, 5, 1, 64, p, None, 0, None)  # noqa
    g = [rows(data=A * (i + 7)) for i in range(3)]
    assert bwd(r[0], r[1], r[2], r[3], r[4], wide, g[1], g[2]) == 1
    assert bwd(r[3], r[1], r[2], r[0], r[4], wide, g[1], g[2]) == 1


def test_heads_past_counting(lib):
    """Counts of heads whose product with the tokens would not fit 64 bits."""
    many = rows(heads=1 << 30, head_stride=0, token_stride=0, batch_stride=0)
    assert fwd(lib, q=many, qo=many, B=1 << 15, N=1 << 15, d=128) == 2


def test_struct_layouts(tmp_path):
    import shutil
    import subprocess
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no host C compiler")
    fields, py = [], []
    for t in (fa.fa_heads_t, fa.fa_norm_rope_t):
        fields.append("sizeof(%s)" % t.__name__)
        py.append(ctypes.sizeof(t))
        for name, _ in t._fields_:
            fields.append("offsetof(%s, %s)" % (t.__name__, name))
            py.append(getattr(t, name).offset)
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "fa.h"\nint main(void) {\n'
                   + "".join('  printf("%%zu ", (size_t)%s);\n' % f for f in fields)
                   + "  return 0;\n}\n")
    exe = tmp_path / "layout"
    subprocess.run([cc, "-I", build.INCLUDE, str(src), "-o", str(exe)], check=True)
    c = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True,
                                        check=True).stdout.split()]
    assert c == py


def test_binding_refuses_host_tensors():
    q = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fa.qk_norm_rope_forward(q, q)
    with pytest.raises(ValueError):
        fa.qk_norm_rope_backward(q, q, q=q, k=q)


def test_binding_refuses_rows_without_tokens(monkeypatch):
    monkeypatch.setattr(fa, "_elsewhere", lambda t: False)
    for shape in ((2, 64), (64,), (1, 1, 2, 3, 64)):
        q = torch.zeros(shape, dtype=torch.bfloat16)
        with pytest.raises(ValueError):
            fa.qk_norm_rope_forward(q, q)
        with pytest.raises(ValueError):
            fa.qk_norm_rope_backward(q, q, norm=False)
