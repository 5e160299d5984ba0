"""The 8-bit cache's and the sampler's entry points without a GPU: every
argument that the header rules out is refused with FDLLM_ERR_ARG and a
message before the device is touched, and the tests' own plain
implementations obey the operators' formulas."""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest
import torch

from kv_cache_decode_dualcache_b200 import build, fdllm
from tests import kv8_ref

P16 = 1 << 20   # an aligned address that nothing dereferences


@pytest.fixture(scope="module")
def lib():
    build.build()
    return fdllm.load_library()


def _cache(**over):
    c = fdllm.FdllmKv8(P16, P16, P16, P16, P16, 0, 0, 0, 8, 2, 4, 4, 128)
    for name, value in over.items():
        setattr(c, name, value)
    return c


def _append_args(**over):
    a = fdllm.FdllmKv8AppendArgs(1, 5, 8, 0, P16, P16, P16, 2048, 128, 2048, 128, 2048, 128, P16,
                                 P16, None, P16, 99, 0, None, None, P16, None, None)
    for name, value in over.items():
        setattr(a, name, value)
    return a


def _attn_args(**over):
    a = fdllm.FdllmKv8AttentionArgs(1, 5, 8, 0, 0, 0.1, P16, 1024, 128, P16, P16, P16, 1024, 128,
                                    None, 0, None)
    for name, value in over.items():
        setattr(a, name, value)
    return a


def _sample_args(**over):
    a = fdllm.FdllmSampleArgs(P16, 100, 0, 4, 100, 99, None, None, None, None, P16, P16, P16)
    for name, value in over.items():
        setattr(a, name, value)
    return a


BAD_CACHES = [dict(k=None), dict(v_scale=None), dict(page_table=None), dict(head_dim=48),
              dict(head_dim=256), dict(n_kv_heads=0), dict(n_seqs=0), dict(n_seqs=65536),
              dict(n_pages=0), dict(max_pages=0), dict(max_pages=(1 << 24) + 1), dict(k=P16 + 8),
              dict(v=P16 + 4), dict(page_stride=4 * 64 * 128 - 16), dict(page_stride=4 * 64 * 128 + 8),
              dict(scale_stride=15), dict(table_stride=3), dict(k_scale=P16 + 2)]


@pytest.mark.parametrize("over", BAD_CACHES, ids=str)
def test_bad_caches_are_refused(lib, over):
    c = _cache(**over)
    for rc in (lib.fdllm_kv8_append(ctypes.byref(c), ctypes.byref(_append_args()), None),
               lib.fdllm_kv8_attention(ctypes.byref(c), ctypes.byref(_attn_args()), None)):
        assert rc == fdllm.FDLLM_ERR_ARG
        assert lib.fdllm_last_error(None).startswith(b"fdllm_kv8_a")


@pytest.mark.parametrize("over", [
    dict(dtype=3), dict(dtype=-1), dict(n_tokens=-1), dict(max_new=-1), dict(reserved=1),
    dict(starts=None), dict(lens=None), dict(k=None), dict(v=None), dict(k=P16 + 8),
    dict(k_token=2044), dict(v_head=4), dict(q_token=2047), dict(q_out=None), dict(q=None),
    dict(n_heads=0), dict(rope_len=0), dict(rope=P16 + 4), dict(k_out=P16 + 2), dict(lens_out=P16),
    dict(status=P16 + 1)], ids=str)
def test_bad_append_arguments_are_refused(lib, over):
    rc = lib.fdllm_kv8_append(ctypes.byref(_cache()), ctypes.byref(_append_args(**over)), None)
    assert rc == fdllm.FDLLM_ERR_ARG and lib.fdllm_last_error(None).startswith(b"fdllm_kv8_append: ")


@pytest.mark.parametrize("over", [
    dict(dtype=3), dict(n_tokens=-1), dict(max_q=-1), dict(max_len=-1), dict(n_heads=6),
    dict(n_heads=0), dict(scale=float("nan")), dict(scale=float("inf")), dict(starts=None),
    dict(lens=None), dict(q=None), dict(out=None), dict(q=P16 + 8), dict(q_token=1025),
    dict(out_head=4), dict(starts=P16 + 2)], ids=str)
def test_bad_attention_arguments_are_refused(lib, over):
    rc = lib.fdllm_kv8_attention(ctypes.byref(_cache()), ctypes.byref(_attn_args(**over)), None)
    assert rc == fdllm.FDLLM_ERR_ARG
    assert lib.fdllm_last_error(None).startswith(b"fdllm_kv8_attention: ")


@pytest.mark.parametrize("over", [dict(out=P16 * 2, out_token=0), dict(out=P16 * 2, out_head=0), dict(),
                                  dict(out=P16 * 2, out_token=64), dict(out=P16 * 2, out_head=-64)], ids=str)
def test_attention_outputs_that_share_memory_are_refused(lib, over):
    """Rows or heads of out on top of one another (an expanded tensor), and out on
    q, whose rows other CTAs may still read."""
    rc = lib.fdllm_kv8_attention(ctypes.byref(_cache()), ctypes.byref(_attn_args(**over)), None)
    assert rc == fdllm.FDLLM_ERR_ARG and b"overlap" in lib.fdllm_last_error(None)


@pytest.mark.parametrize("tokens,heads", [(0x7fffffff, 4), (0x7fffff01, 4), (0x3fffffc0, 8)])
def test_query_rows_beyond_the_kernels_indices_are_refused(lib, tokens, heads):
    """Tiles of up to 256 rows are counted in 32 bits."""
    a = _attn_args(out=2 * P16, n_tokens=tokens, n_heads=heads)
    assert lib.fdllm_kv8_attention(ctypes.byref(_cache()), ctypes.byref(a), None) == fdllm.FDLLM_ERR_ARG
    assert b"query rows" in lib.fdllm_last_error(None)


@pytest.mark.parametrize("over", [dict(lens_out=P16 + 4), dict(lens_out=P16 + 8), dict(lens_out=P16 - 4),
                                  dict(lens=P16 + 64, lens_out=P16 + 68), dict(pos=P16 + 64, lens_out=P16 + 60)], ids=str)
def test_append_lens_out_over_its_inputs_is_refused(lib, over):
    """Two sequences: starts are 3 words, lens and pos 2 each; other CTAs may read
    them after lens_out has been written."""
    a = _append_args(**over)
    assert lib.fdllm_kv8_append(ctypes.byref(_cache()), ctypes.byref(a), None) == fdllm.FDLLM_ERR_ARG
    assert b"lens_out" in lib.fdllm_last_error(None)


@pytest.mark.parametrize("over", [
    dict(dtype=7), dict(rows=-1), dict(vocab=0), dict(vocab=(1 << 18) + 1, row_stride=1 << 20),
    dict(row_stride=99), dict(mask_id=100), dict(mask_id=-2), dict(logits=None), dict(u=None),
    dict(tok=None), dict(logits=P16 + 2), dict(u=P16 + 4), dict(top_k=P16 + 1)], ids=str)
def test_bad_sample_arguments_are_refused(lib, over):
    assert lib.fdllm_sample(ctypes.byref(_sample_args(**over)), None) == fdllm.FDLLM_ERR_ARG
    assert lib.fdllm_last_error(None).startswith(b"fdllm_sample: ")


def test_null_structs_are_refused(lib):
    c, n = _cache(), ctypes.c_size_t()
    assert lib.fdllm_kv8_append(None, ctypes.byref(_append_args()), None) == fdllm.FDLLM_ERR_ARG
    assert lib.fdllm_kv8_append(ctypes.byref(c), None, None) == fdllm.FDLLM_ERR_ARG
    assert lib.fdllm_kv8_attention(ctypes.byref(c), None, None) == fdllm.FDLLM_ERR_ARG
    assert lib.fdllm_kv8_attention_workspace(ctypes.byref(c), None, ctypes.byref(n)) == fdllm.FDLLM_ERR_ARG
    assert lib.fdllm_sample(None, None) == fdllm.FDLLM_ERR_ARG


def test_f16_is_not_a_model_dtype(lib):
    from kv_cache_decode_dualcache_b200 import synth
    cfg = fdllm.make_config(synth.TINY, 96)
    cfg.dtype = 2
    ctx = ctypes.c_void_p()
    assert lib.fdllm_create(ctypes.byref(cfg), 0, None, None, ctypes.byref(ctx)) == fdllm.FDLLM_ERR_ARG


def test_struct_sizes_match_the_header(tmp_path):
    """The binding's structs have the C structs' sizes and last offsets."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = tmp_path / "s.c"
    src.write_text('#include "fdllm.h"\n#include <stdio.h>\n#include <stddef.h>\nint main(void) {'
                   'printf("%zu %zu %zu %zu %zu %zu %zu %zu\\n", sizeof(fdllm_kv8), offsetof(fdllm_kv8, head_dim),'
                   'sizeof(fdllm_kv8_append_args), offsetof(fdllm_kv8_append_args, status),'
                   'sizeof(fdllm_kv8_attention_args), offsetof(fdllm_kv8_attention_args, status),'
                   'sizeof(fdllm_sample_args), offsetof(fdllm_sample_args, prob)); return 0; }')
    exe = tmp_path / "s"
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(root, "include"), str(src), "-o", str(exe)],
                   check=True, timeout=120)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, timeout=60).stdout.split()]
    want = []
    for st, last in ((fdllm.FdllmKv8, "head_dim"), (fdllm.FdllmKv8AppendArgs, "status"),
                     (fdllm.FdllmKv8AttentionArgs, "status"), (fdllm.FdllmSampleArgs, "prob")):
        want += [ctypes.sizeof(st), getattr(st, last).offset]
    assert got == want


def test_constants_match_the_header():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(root, "include", "fdllm.h")).read()
    found = dict(re.findall(r"#define FDLLM_(KV8_\w+) (\d+)", text))
    assert set(found) == {"KV8_PAGE", "KV8_BLOCK", "KV8_BAD_PAGE", "KV8_BAD_RANGE", "KV8_TIMEOUT"}
    assert {n: getattr(fdllm, n) for n in found} == {n: int(v) for n, v in found.items()}


def test_binding_refuses_cpu_tensors_and_wrong_shapes():
    c = kv8_ref.make_cache(torch.Generator().manual_seed(0), [5], 2, 64)
    with pytest.raises(ValueError, match="CUDA"):
        fdllm.Kv8Cache(c["k"], c["v"], c["k_scale"], c["v_scale"], c["table"])
    with pytest.raises(ValueError, match="int8"):
        fdllm.Kv8Cache(c["k"].float(), c["v"], c["k_scale"], c["v_scale"], c["table"])
    with pytest.raises(ValueError, match="CUDA"):
        fdllm.fdllm_sample(torch.zeros(2, 5), torch.zeros(2, dtype=torch.float64))


def test_overlapping_cache_rows_are_refused():
    """An expanded page table (one context for several sequences), pool or scales
    have a row stride of 0, which the C struct takes for dense rows: reads past
    the storage.  Rows that overlap otherwise are refused alike."""
    k, s = torch.zeros(3, 2, 64, 32, dtype=torch.int8), torch.zeros(3, 2, 4)
    table = torch.zeros(4, 8, dtype=torch.int32)
    wide = torch.zeros(100, dtype=torch.int32)
    for over in (dict(table=table[:1].expand(4, -1)), dict(table=wide.as_strided((4, 8), (7, 1))),
                 dict(table=wide[:1].as_strided((4, 1), (0, 0))),
                 dict(k=k[:1].expand(3, -1, -1, -1), v=k[:1].expand(3, -1, -1, -1)),
                 dict(ks=s[:1].expand(3, -1, -1), vs=s[:1].expand(3, -1, -1))):
        a = dict(k=k, v=k, ks=s, vs=s, table=table) | over
        with pytest.raises(ValueError, match="overlap"):
            fdllm.Kv8Cache(*a.values())
    # one row or page: its stride says nothing; rows that only touch are dense
    for table in (wide[:8].expand(1, -1), wide.as_strided((4, 8), (8, 1)), wide.as_strided((4, 1), (1, 1))):
        with pytest.raises(ValueError, match="CUDA"):
            fdllm.Kv8Cache(k, k, s, s, table)
    with pytest.raises(ValueError, match="CUDA"):
        fdllm.Kv8Cache(k[:1].expand(1, -1, -1, -1), k[:1], s[:1], s[:1], wide[:8].view(1, 8))


def test_the_library_is_built_without_its_python_binding(tmp_path, monkeypatch):
    """A machine whose torch headers or g++ do not fit still gets libfdllm.so; the
    operators then say why they are missing.  A binding of another torch is
    built anew, and not left in place when that fails."""
    made = []
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libfdllm.so"))
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_binding.so"))
    monkeypatch.setattr(build, "BINDING_STAMP", str(tmp_path / "stamp"))
    monkeypatch.setattr(build, "build_library", lambda lib, *a: made.append(lib) or lib)
    run = subprocess.run

    def no_gxx(cmd, *a, **kw):
        if cmd[0] == "g++":
            return subprocess.CompletedProcess(cmd, 1, b"no headers", b"")
        return run(cmd, *a, **kw)

    monkeypatch.setattr(build.subprocess, "run", no_gxx)
    (tmp_path / "_binding.so").write_bytes(b"of another torch")
    with pytest.warns(RuntimeWarning, match="no headers"):
        assert build.build() == build.LIB
    assert made == [build.LIB] and not os.path.exists(build.BINDING)
    with pytest.raises(RuntimeError, match="no headers"):
        build.build_binding()
    # built, then found up to date; another torch's stamp: built again
    calls = []

    def gxx(cmd, *a, **kw):
        calls.append(cmd)
        open(cmd[cmd.index("-o") + 1], "wb").close()
        return subprocess.CompletedProcess(cmd, 0, b"", b"")

    monkeypatch.setattr(build.subprocess, "run", gxx)
    build.build_binding()
    build.build_binding()
    assert len(calls) == 1 and os.path.exists(build.BINDING)
    monkeypatch.setattr(torch, "__version__", "0.0")
    build.build_binding()
    assert len(calls) == 2


# ------------------------------------------------ the plain implementations
def test_plain_append_keeps_values_within_half_a_step():
    g = torch.Generator().manual_seed(1)
    lens, n = [13, 0, 64], [9, 33, 1]
    cache = kv8_ref.make_cache(g, [a + b for a, b in zip(lens, n)], 2, 32)
    before = {w: [kv8_ref.dense(cache, w, i, L) for i, L in enumerate(lens)] for w in "kv"}
    x = torch.randn(sum(n), 2, 32, generator=g)
    starts = [0, 9, 42, 43]
    out = kv8_ref.append(cache, x, 3 * x, starts, lens)
    assert out["lens"] == [22, 33, 65]
    for w, y in (("k", x), ("v", 3 * x)):
        for i, L in enumerate(lens):
            now = kv8_ref.dense(cache, w, i, L + n[i])
            pages = cache["table"][i, :-(-(L + n[i]) // 64)].long()
            step = cache[w + "_scale"][pages].double().repeat_interleave(16, 2)[..., None]
            step = step.transpose(0, 1).flatten(1, 2)[:, :L + n[i]]
            new = y[starts[i]:starts[i + 1]].transpose(0, 1).double()
            assert ((now[:, L:] - new).abs() <= step[:, L:] * 0.5000005).all()
            assert ((now[:, :L] - before[w][i]).abs() <= step[:, :L] * 0.5000005).all()


def test_plain_sampler_special_cases():
    z = [0.0, 2.0, 2.0, -1.0, 5.0]
    # mask id out, greedy takes the lower id of equal logits; its share is the softmax's
    tok, prob, _ = kv8_ref.sample_row(z, 0.5, temperature=0.0, mask_id=4)
    e = np.exp(np.array(z[:4]) - 2)
    assert tok == 1 and prob == pytest.approx(1 / e.sum(), rel=1e-14)
    # u walks the ids in order
    c = np.cumsum(np.exp(np.array(z) - 5)) / np.exp(np.array(z) - 5).sum()
    for i in range(5):
        lo = c[i - 1] if i else 0.0
        assert kv8_ref.sample_row(z, (lo + c[i]) / 2)[0] == i
    assert kv8_ref.sample_row(z, 0.999, top_k=2)[2] == [1, 4]
    assert kv8_ref.sample_row(z, 0.999, top_k=2, mask_id=4)[2] == [1, 2]
    assert kv8_ref.sample_row([1.0, 1.0, 1.0, 1.0], 0.9, top_p=0.5)[2] == [0, 1]
    assert kv8_ref.sample_row(z, 0.1, top_p=0.0)[2] == [4]
    assert kv8_ref.sample_row(z, 0.1, min_p=float(np.exp(-3)) * 0.999)[2] == [1, 2, 4]
    assert kv8_ref.sample_row([float("nan"), -np.inf], 0.1) == (-1, 0.0, [])
    assert kv8_ref.sample_row([np.inf, 0.0, np.inf], 0.6)[0] == 2
