"""Rotation plans and argument checks of the generation entry points (CPU:
nothing is enqueued)."""
import ctypes
import math
import os
import subprocess

import pytest
import torch

import generation_ref as ref

INVALID, UNSUP = 1, 2
BIG = 1 << 40


@pytest.fixture(scope="module")
def attn():
    from attention_attn_fwd_04_gb300 import build as b
    b.build()
    import attention_attn_fwd_04_gb300 as a
    return a


@pytest.mark.parametrize("kw", [
    dict(), dict(base=500000.0), dict(scaling="linear", factor=4.0),
    dict(scaling="ntk", factor=8.0), dict(scaling="yarn", factor=4.0, original_len=4096),
    dict(scaling="yarn", factor=16.0, original_len=100, beta_fast=2.0, beta_slow=1.9),
    dict(scaling="yarn", factor=1.0, original_len=8192),
    dict(scaling="bands", factor=8.0, original_len=8192),
    dict(scaling="bands", factor=2.0, original_len=64, low_factor=2.0, high_factor=2.5)])
@pytest.mark.parametrize("rot", [4, 64, 128, 256])
def test_plan_frequencies(attn, kw, rot):
    p = attn.rope_plan(rot, layout="interleaved", **kw)
    want, m = ref.freqs(rot, **kw)
    assert p.rot_dim == rot and p.layout == "interleaved"
    assert p.mscale == pytest.approx(m, rel=2.0 ** -23)
    for a, b in zip(p.inv_freq(), want):
        assert a == pytest.approx(b, rel=1e-14, abs=1e-18)


def test_plan_own_frequencies_wrap_to_turns(attn):
    # frequencies of a turn or more, negative and tiny ones, modulo one turn
    inv = [7.0, -0.5, 0.0, 2 * math.pi, 1e-30, -1e-300]
    p = attn.rope_plan(12, inv_freq=inv)
    got = p.inv_freq()
    tau = 2 * math.pi
    for a, b in zip(got, inv):
        d = (a - b) % tau
        assert min(d, tau - d) <= 1e-14
    assert p.mscale == 1.0


@pytest.mark.parametrize("rot,kw", [
    (0, {}), (3, {}), (258, {}), (-2, {}), (64, dict(base=1.0)), (64, dict(base=-5.0)),
    (64, dict(base=float("nan"))), (64, dict(scaling="linear", factor=0.5)),
    (64, dict(scaling="linear", factor=float("inf"))), (2, dict(scaling="ntk", factor=2.0)),
    (64, dict(scaling="yarn", factor=2.0)), (64, dict(scaling="bands", factor=2.0)),
    (64, dict(scaling="yarn", factor=2.0, original_len=100, beta_fast=1.0, beta_slow=1.0)),
    (64, dict(scaling="yarn", factor=2.0, original_len=100, beta_slow=-1.0)),
    (64, dict(scaling="bands", factor=2.0, original_len=100, low_factor=4.0)),
    (64, dict(mscale=float("inf"))), (64, dict(mscale=1e39)),
    (4, dict(inv_freq=[1.0, float("nan")])), (4, dict(scaling="ntk", factor=1e300))])
def test_plan_refusals(attn, rot, kw):
    with pytest.raises(attn.AttnError) as e:
        attn.rope_plan(rot, **kw)
    assert e.value.status == INVALID


@pytest.mark.parametrize("kw", [dict(layout="quarter"), dict(scaling="dynamic"),
                                dict(inv_freq=[1.0]), dict(inv_freq=[1.0] * 32, scaling="ntk"),
                                dict(mscale=0.0), dict(mscale=-1.0)])
def test_plan_binding_refusals(attn, kw):
    with pytest.raises(ValueError):
        attn.rope_plan(64, **kw)


@pytest.mark.parametrize("kw", [
    dict(base=0.0), dict(base=0, scaling="linear", factor=2.0),
    dict(scaling="yarn", factor=2.0, original_len=100, beta_fast=0.0),
    dict(scaling="yarn", factor=2.0, original_len=100, beta_slow=0),
    dict(scaling="bands", factor=2.0, original_len=100, low_factor=0.0),
    dict(scaling="bands", factor=2.0, original_len=100, high_factor=0.0)])
def test_plan_takes_no_zero_for_a_default(attn, kw):
    # 0 stands for the default in attn_rope_config only
    with pytest.raises(ValueError):
        attn.rope_plan(64, **kw)
    # what a scaling does not read may be anything
    attn.rope_plan(64, beta_fast=0.0, low_factor=0.0)
    attn.rope_plan(4, inv_freq=[1.0, 0.5], base=0.0)


def arr(*v):
    return (ctypes.c_int64 * len(v))(*v)


def plan(attn, rot=64):
    return attn.rope_plan(rot)


def rope_call(attn, x=BIG, xs=(2048, 1024, 64), out=2 * BIG, os_=(2048, 1024, 64), B=2, H=2, S=16,
              D=64, pos=3 * BIG, ps=16, p=None, fn="attn_rope"):
    pl = plan(attn) if p is None else p
    return getattr(attn.lib(), fn)(x, arr(*xs) if xs else None, out, arr(*os_) if os_ else None, B,
                                   H, S, D, pos, ps, 0, pl._ref if pl else None, None)


@pytest.mark.parametrize("fn", ["attn_rope", "attn_rope_bwd"])
@pytest.mark.parametrize("kw,want", [
    (dict(x=None), INVALID), (dict(out=None), INVALID), (dict(xs=None), INVALID),
    (dict(B=0), INVALID), (dict(S=-1), INVALID), (dict(D=63), INVALID), (dict(D=32), INVALID),
    (dict(D=2048), UNSUP), (dict(x=BIG + 1), INVALID), (dict(pos=BIG + 2), INVALID),
    (dict(ps=-1), INVALID), (dict(xs=(2048, 1024, -64)), INVALID),
    (dict(os_=(2048, 1024, 0)), INVALID), (dict(os_=(2048, 1024, 32)), INVALID),
    (dict(os_=(1024, 1024, 64)), INVALID), (dict(out=BIG + 64), INVALID),
    (dict(out=BIG, os_=(2048, 64, 128)), INVALID), (dict(pos=2 * BIG), INVALID),
    (dict(B=1 << 16, S=1 << 16), INVALID), (dict(xs=(1 << 62, 1 << 62, 64)), INVALID),
    (dict(p=False), INVALID)])
def test_rope_refusals(attn, kw, want, fn):
    assert rope_call(attn, fn=fn, **kw) == want


def test_rope_plan_struct_refusals(attn):
    for field, value in (("version", 2), ("rot_dim", 0), ("rot_dim", 7), ("rot_dim", 512),
                         ("layout", 2), ("mscale", float("nan"))):
        p = plan(attn)
        setattr(p._struct, field, value)
        assert rope_call(attn, p=p) == INVALID


def desc(attn, **kw):
    from attention_attn_fwd_04_gb300.generation import CacheDesc
    d = CacheDesc(1, 0, 10, 16, 2, 64, 5 * BIG, 6 * BIG, (2048, 1024, 64), (2048, 1024, 64))
    for k, v in kw.items():
        setattr(d, k, (ctypes.c_int64 * 3)(*v) if isinstance(v, tuple) else v)
    return d


BAD_CACHES = [
    (dict(version=0), INVALID), (dict(dtype=2), INVALID), (dict(num_pages=0), INVALID),
    (dict(page_size=0), INVALID), (dict(H_kv=0), INVALID), (dict(D=0), INVALID),
    (dict(D=96), UNSUP), (dict(k=None), INVALID), (dict(k=5 * BIG + 8), INVALID),
    (dict(k_strides=(2048, 1024, 60)), INVALID), (dict(k_strides=(2048, 1024, 68)), INVALID),
    (dict(v_strides=(1024, 1024, 64)), INVALID), (dict(v_strides=(2048, 1024, 0)), INVALID),
    (dict(k_strides=(-2048, 1024, 64)), INVALID), (dict(k_scale=BIG), INVALID),
    (dict(dtype=1, k_strides=(2048, 1024, 72)), INVALID), (dict(dtype=1, v_scale=BIG + 1), INVALID)]


def append_call(attn, q=BIG, qs=(512, 64), k=2 * BIG, ks=(512, 64), v=3 * BIG, vs=(512, 64),
                qo=4 * BIG, qos=(512, 64), T=8, H=4, pos=7 * BIG, slots=8 * BIG, p=None, d=None):
    pl = plan(attn) if p is None else p
    d = desc(attn) if d is None else d
    return attn.lib().attn_cache_append(
        q, arr(*qs) if qs else None, k, arr(*ks), v, arr(*vs), qo, arr(*qos) if qos else None, T, H,
        pos, slots, pl._ref if pl else None, ctypes.byref(d) if d is not False else None, None)


@pytest.mark.parametrize("kw,want", [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(slots=None), INVALID),
    (dict(qo=None), INVALID), (dict(q=None), INVALID), (dict(qs=None), INVALID),
    (dict(T=0), INVALID), (dict(T=(1 << 24) + 1), INVALID), (dict(H=0), INVALID),
    (dict(H=70000, qs=(70000 * 64, 64), qos=(70000 * 64, 64)), INVALID),
    (dict(pos=None), INVALID), (dict(p=False), INVALID), (dict(slots=BIG + 4), INVALID),
    (dict(k=5 * BIG), INVALID), (dict(v=6 * BIG + 128), INVALID), (dict(slots=6 * BIG), INVALID),
    (dict(qo=2 * BIG), INVALID), (dict(qo=BIG + 64), INVALID), (dict(qo=5 * BIG), INVALID),
    (dict(qo=7 * BIG), INVALID), (dict(qos=(64, 64)), INVALID), (dict(d=False), INVALID),
    # in place, but q is k too
    (dict(qo=BIG, k=BIG), INVALID),
    # in place, and keys lie in the queries' part of the tokens
    (dict(qo=BIG, k=BIG + 2 * 192), INVALID)])
def test_append_refusals(attn, kw, want):
    assert append_call(attn, **kw) == want


@pytest.mark.parametrize("kw,want", BAD_CACHES + [(dict(v=5 * BIG), INVALID)])  # v is k
def test_append_cache_refusals(attn, kw, want):
    assert append_call(attn, d=desc(attn, **kw)) == want


def slots_call(attn, ctx=BIG, new=2 * BIG, B=4, page=16, pages=10, table=3 * BIG, ts=8, mp=8,
               free=4 * BIG, cap=10, nf=5 * BIG, seq=6 * BIG, cu=7 * BIG, req=8 * BIG, pos=9 * BIG,
               slots=10 * BIG, nfo=11 * BIG, T=32):
    return attn.lib().attn_cache_slots(ctx, new, B, page, pages, table, ts, mp, free, cap, nf, seq,
                                       cu, req, pos, slots, nfo, T, None)


@pytest.mark.parametrize("kw,want", [
    (dict(ctx=None), INVALID), (dict(slots=None), INVALID), (dict(table=None), INVALID),
    (dict(B=0), INVALID), (dict(B=16385), UNSUP), (dict(page=0), INVALID), (dict(pages=0), INVALID),
    (dict(mp=0), INVALID), (dict(ts=7), INVALID), (dict(T=0), INVALID),
    (dict(T=(1 << 30) + 1), INVALID), (dict(mp=1 << 27, ts=1 << 27), INVALID),
    (dict(nf=None), INVALID), (dict(nfo=None), INVALID), (dict(cap=-1), INVALID),
    (dict(free=None), INVALID), (dict(ctx=BIG + 2), INVALID), (dict(slots=10 * BIG + 4), INVALID),
    (dict(seq=2 * BIG), INVALID), (dict(seq=BIG + 4), INVALID), (dict(cu=BIG), INVALID),
    (dict(req=9 * BIG), INVALID), (dict(pos=10 * BIG), INVALID), (dict(table=4 * BIG), INVALID),
    (dict(nfo=4 * BIG + 8), INVALID), (dict(slots=3 * BIG + 64), INVALID)])
def test_slots_refusals(attn, kw, want):
    assert slots_call(attn, **kw) == want


def decode_call(attn, q=BIG, qs=(256, 64), d=None, table=2 * BIG, ts=8, mp=8, lens=3 * BIG,
                out=4 * BIG, lse=7 * BIG, B=2, H=4, scale=0.125, mod=None, ws=8 * BIG, wsb=1 << 30):
    d = desc(attn) if d is None else d
    return attn.lib().attn_decode(q, arr(*qs) if qs else None,
                                  ctypes.byref(d) if d is not False else None, table, ts, mp, lens,
                                  out, lse, B, H, scale, ctypes.byref(mod) if mod else None, ws, wsb,
                                  None)


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), INVALID), (dict(qs=None), INVALID), (dict(d=False), INVALID),
    (dict(table=None), INVALID), (dict(lens=None), INVALID), (dict(out=None), INVALID),
    (dict(ws=None), INVALID), (dict(wsb=100), INVALID), (dict(ws=8 * BIG + 8), INVALID),
    (dict(B=0), INVALID), (dict(B=65537), INVALID), (dict(H=3), INVALID), (dict(H=0), INVALID),
    (dict(H=65536), INVALID), (dict(mp=0), INVALID), (dict(mp=1 << 27), INVALID),
    (dict(scale=0.0), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(ts=-1), INVALID), (dict(q=BIG + 2), INVALID),
    (dict(qs=(255, 64)), INVALID), (dict(qs=(256, -64)), INVALID), (dict(out=4 * BIG + 8), INVALID),
    (dict(lse=7 * BIG + 2), INVALID), (dict(out=BIG), INVALID), (dict(out=5 * BIG), INVALID),
    (dict(lse=4 * BIG), INVALID), (dict(ws=4 * BIG), INVALID), (dict(ws=6 * BIG), INVALID),
    (dict(lse=3 * BIG), INVALID),
    (dict(B=65536, H=32768, ts=0, mp=1 << 26, qs=(0, 0)), UNSUP)])
def test_decode_refusals(attn, kw, want):
    assert decode_call(attn, **kw) == want


@pytest.mark.parametrize("kw,want", BAD_CACHES)
def test_decode_cache_refusals(attn, kw, want):
    assert decode_call(attn, d=desc(attn, **kw)) == want


def test_outputs_beside_scales_slopes_and_biases(attn):
    # every array that a call reads while others of its CTAs already write
    def modded(score_flags, **kw):
        m = attn.ModDesc()
        m.version, m.score_flags = 2, score_flags
        for k, v in kw.items():
            setattr(m, k, v)
        return m
    for out, size in (("out", 2 * 4 * 64 * 2), ("lse", 2 * 4 * 4), ("ws", 1 << 30)):
        base = dict(out=4 * BIG, lse=7 * BIG, ws=8 * BIG)[out]
        for at in (base, base + size - 4):
            for f in ("k_scale", "v_scale"):
                assert decode_call(attn, d=desc(attn, dtype=1, **{f: at})) == INVALID
            assert decode_call(attn, mod=modded(attn.SCORE_ALIBI, alibi_slopes=at)) == INVALID
            assert decode_call(attn, mod=modded(attn.SCORE_RELBIAS, rel_bias=at, rel_max=3)) == INVALID
        # the last of H (2 R + 1) biases
        assert decode_call(attn, mod=modded(attn.SCORE_RELBIAS, rel_bias=base - 4 * (4 * 7 - 1),
                                            rel_max=3)) == INVALID
    for f in ("k_scale", "v_scale"):
        for at in (5 * BIG, 6 * BIG + 64, 4 * BIG + 4 * 64 * 2):
            assert append_call(attn, d=desc(attn, dtype=1, **{f: at})) == INVALID


def test_decode_mod_refusals(attn):
    def with_mod(version=2, **kw):
        m = attn.ModDesc()
        m.version = version
        for k, v in kw.items():
            setattr(m, k, v)
        return decode_call(attn, mod=m)
    assert with_mod(version=7) == INVALID
    assert with_mod(mask_flags=attn.MASK_WINDOW, window=0) == INVALID
    assert with_mod(score_flags=attn.SCORE_SOFTCAP, softcap=-1.0) == INVALID
    assert with_mod(score_flags=attn.SCORE_RELBIAS) == INVALID
    assert with_mod(mask_flags=1 << 9) == INVALID
    assert with_mod(mask_flags=attn.MASK_DOCUMENT, doc_ids=BIG) == UNSUP
    assert with_mod(mask_flags=attn.MASK_PREFIX_LM, prefix_len=BIG) == UNSUP
    assert with_mod(mask_flags=attn.MASK_BLOCKS, blocks=BIG) == UNSUP
    assert with_mod(q_offset=1) == UNSUP
    assert with_mod(block_mask=BIG) == UNSUP


def test_decode_workspace_bytes(attn):
    n = attn.decode_workspace_bytes
    assert n(32, 8, 128) > 0 and n(32, 8, 128) % 16 == 0
    assert n(16, 1, 128) > n(8, 1, 128)   # 16 query heads a part instead of 8
    for bad in ((0, 1, 64), (4, 0, 64), (4, 3, 64), (4, 4, 96), (65536, 1, 64)):
        assert n(*bad) == 0


def test_binding_refuses_cpu_tensors_and_wrong_forms(attn):
    x = torch.zeros((1, 2, 3, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        attn.rope(x, plan(attn))
    with pytest.raises(ValueError):
        attn.cache_append(x[0], x[0], x, x, torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError):
        attn.attn_decode(x[0], x, x, torch.zeros((2, 1), dtype=torch.int32),
                         torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        i = torch.zeros(2, dtype=torch.int32)
        attn.cache_slots(i, i, torch.zeros((2, 1), dtype=torch.int32), page_size=1, num_pages=1,
                         max_tokens=1)


def test_structs_match_the_header(attn, tmp_path):
    """Sizes and offsets of the ctypes mirrors against the C compiler's."""
    from attention_attn_fwd_04_gb300 import generation as g
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    pairs = [("attn_rope_config", g.RopeConfig), ("attn_rope_plan", g.RopePlanStruct),
             ("attn_cache_desc", g.CacheDesc)]
    lines = []
    for name, cls in pairs:
        lines.append('printf("%%zu\\n", sizeof(%s));' % name)
        lines += ['printf("%%zu\\n", offsetof(%s, %s));' % (name, f[0]) for f in cls._fields_]
    src = tmp_path / "s.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "attn.h"\n'
                   "int main(void) { %s return 0; }\n" % " ".join(lines))
    exe = tmp_path / "s"
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-pedantic", "-I",
                    os.path.join(root, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], check=True, capture_output=True,
                                          text=True).stdout.split()]
    want = []
    for _, cls in pairs:
        want.append(ctypes.sizeof(cls))
        want += [getattr(cls, f[0]).offset for f in cls._fields_]
    assert got == want


def test_missing_native_module_fails_loudly():
    # no fallback: without the compiled binding the first call raises
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = (
        "import sys, torch\n"
        "import attention_attn_fwd_04_gb300 as a\n"
        "sys.modules['attention_attn_fwd_04_gb300._generation'] = None\n"
        "try:\n"
        "    a.rope(torch.zeros(1), a.rope_plan(4))\n"
        "except ImportError as e:\n"
        "    print('raised', 'not built' in str(e))\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True,
                       timeout=300)
    assert "raised True" in r.stdout, r.stdout + r.stderr


def test_native_module_argument_types(attn):
    from attention_attn_fwd_04_gb300 import generation as g
    x = torch.zeros((1, 2, 3, 64), dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        attn.rope([1, 2], plan(attn))            # not a tensor
    for fn in (g._native.rope, g._native.slots, g._native.append, g._native.decode):
        with pytest.raises(TypeError):
            fn(x)                                # wrong number of arguments


def test_binding_is_rebuilt_for_another_torch_or_python(attn, monkeypatch):
    # the module inlines accessors of one torch version: a change of torch (or
    # of the interpreter) has to rebuild it though no source is newer
    import sysconfig

    from attention_attn_fwd_04_gb300 import build as b
    from attention_attn_fwd_04_gb300 import _generation
    assert os.path.samefile(_generation.__file__, b.BINDING)
    assert b.BINDING.endswith(sysconfig.get_config_var("EXT_SUFFIX"))
    assert not os.path.exists(os.path.join(b.HERE, "_generation.so"))
    made = []
    monkeypatch.setattr(b, "_compile_binding", lambda obj: made.append("compiled") or "")
    monkeypatch.setattr(b, "_link_binding", lambda obj: made.append("linked"))
    b.build()
    assert made == []
    real = sysconfig.get_config_var
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", "2.9.1+other")
        b.build()
    assert made == ["compiled", "linked"]
    with monkeypatch.context() as m:
        m.setattr(sysconfig, "get_config_var",
                  lambda n: "cpython-313-x86_64-linux-gnu" if n == "SOABI" else real(n))
        b.build()
    assert made == ["compiled", "linked"] * 2
    b.build()
    assert made == ["compiled", "linked"] * 2
