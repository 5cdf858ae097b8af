"""The tree operators' C ABI without a GPU: struct layouts, packed formats, host checks."""
import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROBE = r"""
#include <stddef.h>
#include <stdio.h>
#include "specdec.h"
#define F(T, f) printf(#T "." #f " %zu\n", offsetof(T, f));
int main(void) {
  printf("max_tree %d\n", SPECDEC_MAX_TREE);
  %FIELDS%
  return 0;
}
"""


def structs(sd):
    return {"specdec_rotary_args": (sd.RotaryArgs, sd._PACK_ROTARY),
            "specdec_tree_attention_args": (sd.TreeAttentionArgs, sd._PACK_ATTENTION),
            "specdec_tree_commit_args": (sd.TreeCommitArgs, sd._PACK_COMMIT)}


def test_struct_layouts(tmp_path):
    import speculative_decoding_specdec_gb300.specdec as sd
    lines = []
    for cn, (py, _) in structs(sd).items():
        lines.append(f'printf("{cn} %zu\\n", sizeof({cn}));')
        lines += [f"F({cn}, {f})" for f, _ in py._fields_]
    src, exe = tmp_path / "probe.c", tmp_path / "probe"
    src.write_text(PROBE.replace("%FIELDS%", "\n".join(lines)))
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    out = dict(x.rsplit(" ", 1) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split("\n") if x)
    assert int(out["max_tree"]) == sd.MAX_TREE
    for cn, (py, _) in structs(sd).items():
        assert int(out[cn]) == ctypes.sizeof(py), cn
        for f, _ in py._fields_:
            assert int(out[f"{cn}.{f}"]) == getattr(py, f).offset, (cn, f)


def test_packed_formats_fill_the_structs():
    import speculative_decoding_specdec_gb300.specdec as sd
    for cn, (py, fmt) in structs(sd).items():
        values = list(range(1, len(fmt.unpack(bytes(fmt.size))) + 1))
        got, at = py.from_buffer_copy(fmt.pack(*values).ljust(ctypes.sizeof(py), b"\0")), iter(values)
        assert ctypes.sizeof(py) - fmt.size < 8, cn          # trailing padding only
        for f, t in py._fields_:
            v = getattr(got, f)
            for x in ([getattr(v, g) for g, _ in t._fields_] if t is sd.KvView else [v]):
                assert x == next(at), (cn, f)
        assert next(at, None) is None


def test_host_checks():
    import speculative_decoding_specdec_gb300.specdec as sd
    L = sd.lib
    for f in (L.specdec_rotary_append, L.specdec_tree_attention, L.specdec_tree_commit):
        assert f(None, None) == sd.ERR_INVALID_ARG
    r = sd.RotaryArgs(B=0, T=1, heads_q=1, table_len=1)
    assert L.specdec_rotary_append(ctypes.byref(r), None) == sd.OK
    r.B = 1
    assert L.specdec_rotary_append(ctypes.byref(r), None) == sd.ERR_INVALID_ARG      # no cache
    a = sd.TreeAttentionArgs(B=0, T=1, heads_q=1, scale=1.0)
    assert L.specdec_tree_attention(ctypes.byref(a), None) == sd.OK
    for kw, code in ((dict(T=0), sd.ERR_INVALID_ARG), (dict(T=65), sd.ERR_UNSUPPORTED), (dict(B=1025), sd.ERR_UNSUPPORTED),
                     (dict(scale=float("nan")), sd.ERR_INVALID_ARG), (dict(B=1), sd.ERR_INVALID_ARG), (dict(B=-1), sd.ERR_INVALID_ARG)):
        a = sd.TreeAttentionArgs(**({"B": 0, "T": 1, "heads_q": 1, "scale": 1.0} | kw))
        assert L.specdec_tree_attention(ctypes.byref(a), None) == code, kw
    c = sd.TreeCommitArgs(B=0, T=2, D=1)
    assert L.specdec_tree_commit(ctypes.byref(c), None) == sd.OK
    for kw, code in ((dict(T=65), sd.ERR_UNSUPPORTED), (dict(D=32), sd.ERR_UNSUPPORTED), (dict(D=0), sd.ERR_INVALID_ARG), (dict(B=1), sd.ERR_INVALID_ARG)):
        c = sd.TreeCommitArgs(**({"B": 0, "T": 2, "D": 1} | kw))
        assert L.specdec_tree_commit(ctypes.byref(c), None) == code, kw
    fake = 1 << 20
    def greedy(z=fake, dt=sd.BF16, B=1, T=2, V=10, rs=10, D=1, tok=fake):
        return L.specdec_verify_tree_greedy(z, dt, B, T, V, rs, tok, None, D, fake, fake, fake, fake, fake, None)
    def sample(z=fake, w=fake, temp=1.0, B=1, T=2, D=1):
        return L.specdec_verify_tree_sample(z, w, sd.F32, B, T, 10, 10, temp, fake, None, fake, 0, D, fake, fake, fake, fake, fake, None)
    assert greedy(B=0) == sd.OK and sample(B=0) == sd.OK
    for kw in (dict(z=None), dict(z=fake + 1), dict(dt=7), dict(T=0), dict(V=0), dict(rs=9), dict(D=0), dict(tok=None), dict(B=-1)):
        assert greedy(**kw) == sd.ERR_INVALID_ARG, kw
    for kw in (dict(T=65), dict(D=32)):
        assert greedy(**kw) == sd.ERR_UNSUPPORTED and sample(**kw) == sd.ERR_UNSUPPORTED
    for kw in (dict(w=None), dict(w=fake + 2), dict(temp=0.0), dict(temp=float("inf")), dict(temp=float("nan"))):
        assert sample(**kw) == sd.ERR_INVALID_ARG, kw


def test_binding_wants_cuda_tensors():
    import torch
    import speculative_decoding_specdec_gb300.specdec as sd
    cache, q = torch.zeros(1, 2, 1, 2, 4, 8), torch.zeros(1, 1, 2, 8)
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        sd.tree_attention(q, cache, 0, q, i, i, None, i, torch.zeros(256, dtype=torch.uint8))
    with pytest.raises(ValueError):
        sd.rotary_append(q, q, q, cache, 0, torch.zeros(4, 4, 2), q, i, n_committed=i, width=i)
    with pytest.raises(ValueError):
        sd.verify_tree_greedy(torch.zeros(1, 1, 4), i[None], None, i, i, i[None], i[None], i)
    with pytest.raises(ValueError):
        sd.tree_commit(cache, cache, i, i, i[None], i)
