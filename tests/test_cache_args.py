"""CPU tests of the several-axes rotary plan and of every refusal of the cache
operators: all argument checks run on the host before any CUDA call."""
import ctypes

import numpy as np
import pytest
import torch

import joint_text_image_b200 as jt
from joint_text_image_b200 import build as jbuild
from oracle import cache as oc

INVALID, UNSUPPORTED = 1, 2


@pytest.fixture(scope="module", autouse=True)
def built():
    jbuild.build()


@pytest.mark.parametrize("D,n_axes,sections,per_axis", [
    (128, 1, None, False), (128, 2, None, False), (64, 3, None, False), (96, 4, None, False),
    (128, 3, [16, 24, 24], False), (128, 3, [16, 24, 24], True), (64, 2, [0, 32], True), (16, 3, [0, 8, 0], False),
    (256, 4, [1, 2, 3, 122], True), (64, 3, [30, 0, 2], True),
])
def test_plan_matches_the_definition(D, n_axes, sections, per_axis):
    plan = jt.hia_rope_plan(D, n_axes, sections=sections, base=10000.0, per_axis=per_axis)
    ref = oc.rope_pairs(D, n_axes, sections, 10000.0, per_axis)
    assert plan.D == D and plan.n_axes == n_axes and len(ref) == D // 2
    assert [plan.axis[j] for j in range(D // 2)] == [a for a, _ in ref]
    # pow in double: a few units in the last place on either side
    np.testing.assert_allclose([plan.freq[j] for j in range(D // 2)], [f for _, f in ref], rtol=1e-14)


@pytest.mark.parametrize("D,n_axes,sections,base,per_axis", [
    (0, 1, None, 1e4, 0), (24, 1, None, 1e4, 0), (272, 1, None, 1e4, 0), (64, 0, None, 1e4, 0), (64, 5, None, 1e4, 0),
    (64, 2, [16, 15], 1e4, 0), (64, 2, [33, -1], 1e4, 0), (64, 2, None, 0.0, 0), (64, 2, None, -1.0, 0),
    (64, 2, None, float("nan"), 0), (64, 2, None, float("inf"), 0), (64, 2, None, 1e4, 1),
])
def test_plan_refusals(D, n_axes, sections, base, per_axis):
    plan = jt.RopePlan()
    plan.D = 7
    sec = (ctypes.c_int32 * len(sections))(*sections) if sections else None
    assert jt.lib().hia_rope_plan_init(ctypes.byref(plan), D, n_axes, sec, base, per_axis) == INVALID
    assert plan.D == 7, "a refused plan is left as it was"
    assert jt.lib().hia_rope_plan_init(None, 64, 1, None, 1e4, 0) == INVALID


A = 4096  # an aligned address that is never dereferenced


def T_(ptr=A, s=512, hkv=256, hq=64):
    return jt._Tensor(ptr, 0, s, hkv, hq)


NONE = jt._Tensor(None, 0, 0, 0, 0)


def rope_call(plan=None, T=4, pos=A, dtype=0, Hq=8, Hkv=2, q=None, k=None, qo=None, ko=None, fn="fwd"):
    plan = jt.hia_rope_plan(64, 2) if plan is None else plan() if callable(plan) else plan
    f = jt.lib().hia_rope_axes_fwd if fn == "fwd" else jt.lib().hia_rope_axes_bwd
    return f(ctypes.byref(plan) if plan else None, T, pos, dtype, Hq, Hkv, q or T_(), k or T_(), qo or T_(),
             ko or T_(), None)


def bad_plan(**kw):
    p = jt.hia_rope_plan(64, 2)
    for n, v in kw.items():
        if n in ("axis", "freq"):
            getattr(p, n)[5] = v
        else:
            setattr(p, n, v)
    return p


@pytest.mark.parametrize("fn", ["fwd", "bwd"])
@pytest.mark.parametrize("kw,code", [
    (dict(plan=False), INVALID), (dict(T=-1), INVALID), (dict(Hq=0), INVALID), (dict(Hkv=0), INVALID),
    (dict(pos=None), INVALID), (dict(q=NONE), INVALID), (dict(qo=NONE), INVALID), (dict(k=NONE), INVALID),
    (dict(ko=NONE), INVALID), (dict(q=T_(s=-512)), INVALID), (dict(k=T_(hkv=-8)), INVALID),
    (dict(dtype=3), UNSUPPORTED), (dict(dtype=-1), UNSUPPORTED), (dict(Hq=9), UNSUPPORTED),
    (dict(T=1 << 31), UNSUPPORTED), (dict(q=T_(ptr=A + 8)), UNSUPPORTED), (dict(ko=T_(s=516)), UNSUPPORTED),
    (dict(qo=T_(hq=4)), UNSUPPORTED), (dict(k=T_(hkv=12)), UNSUPPORTED),
    (dict(q=T_(s=6), dtype=2), UNSUPPORTED),
    (dict(plan=lambda: bad_plan(axis=2)), INVALID), (dict(plan=lambda: bad_plan(freq=float("nan"))), INVALID),
    (dict(plan=lambda: bad_plan(freq=float("inf"))), INVALID), (dict(plan=lambda: bad_plan(D=72)), INVALID),
    (dict(plan=lambda: bad_plan(n_axes=0)), INVALID), (dict(plan=lambda: bad_plan(n_axes=5)), INVALID),
    (dict(T=0, pos=None, q=NONE, k=NONE, qo=NONE, ko=NONE), 0),
])
def test_rope_refusals(kw, code, fn):
    assert rope_call(fn=fn, **kw) == code


def test_rope_tables_refusals():
    L, plan = jt.lib(), jt.hia_rope_plan(64, 2)
    p = ctypes.byref(plan)
    assert L.hia_rope_axes_tables(None, 1, A, A, A, None) == INVALID
    assert L.hia_rope_axes_tables(p, -1, A, A, A, None) == INVALID
    assert L.hia_rope_axes_tables(p, 1 << 31, A, A, A, None) == UNSUPPORTED
    assert L.hia_rope_axes_tables(p, 1, None, A, A, None) == INVALID
    assert L.hia_rope_axes_tables(p, 1, A, None, A, None) == INVALID
    assert L.hia_rope_axes_tables(p, 1, A, A, None, None) == INVALID
    assert L.hia_rope_axes_tables(p, 0, None, None, None, None) == 0


def cache(**kw):
    c = jt._Cache(A, A, 2 * 64 * 64, 64, 64 * 64, 10, 64, 2, 64, 0)
    for n, v in kw.items():
        setattr(c, n, v)
    return c


def chunk(**kw):
    c = jt._Chunk(A, A, A, 5, 3, 5)
    for n, v in kw.items():
        setattr(c, n, v)
    return c


COMMON = [
    (dict(cache=None), INVALID), (dict(chunk=None), INVALID), (dict(T=-1), INVALID), (dict(Hq=0), INVALID),
    (dict(cache=cache(Hkv=0)), INVALID), (dict(cache=cache(n_pages=-1)), INVALID), (dict(chunk=chunk(B=-1)), INVALID),
    (dict(chunk=chunk(max_pages=-1)), INVALID), (dict(cache=cache(dtype=2)), UNSUPPORTED),
    (dict(cache=cache(dtype=7)), UNSUPPORTED), (dict(cache=cache(D=96)), UNSUPPORTED), (dict(Hq=9), UNSUPPORTED),
    (dict(cache=cache(page_size=8)), UNSUPPORTED), (dict(cache=cache(page_size=48)), UNSUPPORTED),
    (dict(cache=cache(page_size=512)), UNSUPPORTED), (dict(chunk=chunk(max_pages=1 << 24)), UNSUPPORTED),
    (dict(T=1 << 30), UNSUPPORTED), (dict(cache=cache(stride_s=-64)), INVALID),
    (dict(cache=cache(stride_page=-8)), INVALID), (dict(chunk=chunk(page_stride=-1)), INVALID),
    (dict(cache=cache(k=None)), INVALID), (dict(cache=cache(v=None)), INVALID), (dict(cache=cache(n_pages=0)), INVALID),
    (dict(chunk=chunk(rows=None)), INVALID), (dict(chunk=chunk(past=None)), INVALID),
    (dict(chunk=chunk(pages=None)), INVALID), (dict(cache=cache(stride_s=0)), UNSUPPORTED),
    (dict(cache=cache(stride_h=0)), UNSUPPORTED), (dict(cache=cache(stride_page=0)), UNSUPPORTED),
    (dict(cache=cache(k=A + 2)), UNSUPPORTED), (dict(cache=cache(stride_h=68)), UNSUPPORTED),
    (dict(cache=cache(stride_page=8196)), UNSUPPORTED), (dict(chunk=chunk(past=A + 2)), UNSUPPORTED),
    (dict(T=0), 0), (dict(chunk=chunk(B=0)), 0),
]


def ref(x):
    return None if x is None else ctypes.byref(x)


def append_call(cache=cache(), chunk=chunk(), T=4, Hq=8, plan=None, pos=None, norm=None, q=T_(), k=T_(), v=T_(),
                qo=T_()):
    return jt.lib().hia_cache_append(ref(cache), ref(chunk), T, Hq, ref(plan), pos,
                                     ctypes.pointer(norm) if norm else None, q, k, v, qo, None)


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(k=NONE), INVALID), (dict(v=NONE), INVALID), (dict(q=NONE), INVALID), (dict(qo=NONE), INVALID),
    (dict(plan=jt.RopePlan()), INVALID), (dict(k=T_(ptr=A + 2)), UNSUPPORTED), (dict(v=T_(s=4)), UNSUPPORTED),
    (dict(qo=T_(hq=4)), UNSUPPORTED), (dict(norm=jt._QkNorm(None, A, 1e-5)), INVALID),
    (dict(norm=jt._QkNorm(A, None, 1e-5)), INVALID), (dict(norm=jt._QkNorm(A, A, -1.0)), INVALID),
    (dict(norm=jt._QkNorm(A, A, float("nan"))), INVALID), (dict(norm=jt._QkNorm(A, A + 4, 1e-5)), UNSUPPORTED),
])
def test_append_refusals(kw, code):
    assert append_call(**kw) == code


def test_append_plan_refusals():
    assert append_call(plan=jt.hia_rope_plan(128, 2), pos=A) == INVALID  # the cache holds D = 64
    assert append_call(plan=jt.hia_rope_plan(64, 2), pos=None) == INVALID


def attn_call(cache=cache(), chunk=chunk(), T=4, Hq=8, q=T_(), bound=None, scale=0.125, o=T_(), lse=A, ws=A,
              nb=1 << 40):
    return jt.lib().hia_attn_cache_fwd(ref(cache), ref(chunk), T, Hq, q, bound, scale, o, lse, ws, nb, None)


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(q=NONE), INVALID), (dict(o=NONE), INVALID), (dict(ws=None), INVALID),
    (dict(nb=16), INVALID), (dict(ws=A + 16), INVALID), (dict(q=T_(s=-8)), INVALID), (dict(o=T_(ptr=A + 8)), UNSUPPORTED),
    (dict(o=T_(hkv=4)), UNSUPPORTED), (dict(bound=A + 1), UNSUPPORTED), (dict(lse=A + 2), UNSUPPORTED),
    (dict(Hq=2 * 129), UNSUPPORTED),
])
def test_attn_refusals(kw, code):
    assert attn_call(**kw) == code


def test_workspace_bytes():
    L = jt.lib()
    f = lambda c, k, T, Hq: L.hia_attn_cache_workspace_bytes(ref(c), ref(k), T, Hq)
    assert f(cache(), chunk(), 4, 8) > 0
    assert f(cache(), chunk(), 4000, 8) > f(cache(), chunk(), 4, 8)
    for kw, code in COMMON:
        if code:
            a = dict(cache=cache(), chunk=chunk(), T=4, Hq=8)
            a.update(kw)
            assert f(a["cache"], a["chunk"], a["T"], a["Hq"]) == 0


@pytest.mark.parametrize("shared", [dict(s=0), dict(hkv=0), dict(hq=0)])
def test_outputs_that_share_memory(shared):
    """An output (or the attention's q, which is read as boxes) whose rows or
    heads lie on one another; a stride that nothing steps by may be 0."""
    out = T_(**shared)
    assert rope_call(qo=out) == UNSUPPORTED
    assert append_call(qo=out) == UNSUPPORTED
    assert attn_call(o=out) == UNSUPPORTED and attn_call(q=out) == UNSUPPORTED
    if "hq" not in shared:
        assert rope_call(ko=out) == UNSUPPORTED
    # (refused for the workspace, so after the tensors were accepted)
    free = dict(s=dict(T=1), hkv=dict(Hq=4, cache=cache(Hkv=1)), hq=dict(Hq=2))[next(iter(shared))]
    assert attn_call(q=out, o=out, nb=16, **free) == INVALID


def test_status_string():
    assert b"chunk" in jt.lib().hia_status_string(7)


def test_binding_refuses_host_tensors_and_shapes():
    t = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    pos = torch.zeros(4, 2, dtype=torch.int32)
    plan = jt.hia_rope_plan(64, 2)
    with pytest.raises(ValueError):
        jt.hia_rope_axes_fwd(plan, pos, t)            # not on a GPU
    with pytest.raises(ValueError):
        jt.hia_rope_axes_fwd(plan, pos.long(), t)     # positions of another type
    with pytest.raises(ValueError):
        jt.hia_rope_axes_tables(plan, pos[:, :1])     # one axis for a plan of two
    with pytest.raises(ValueError):
        jt.hia_rope_plan(64, 3, sections=[16, 16])    # sections of two axes
    pages = torch.zeros(3, 16, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        jt.hia_cache(pages, pages)
    with pytest.raises(ValueError):
        jt.Cache(pages, pages[:2])
    with pytest.raises(ValueError):
        jt.Cache(pages, pages.half())
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    with pytest.raises(ValueError):
        jt.Chunk(i32(2, 3), i32(2), i32(2))           # rows: B + 1
    with pytest.raises(ValueError):
        jt.Chunk(i32(3, 3), i32(2), i32(3))
    with pytest.raises(ValueError):
        jt.Chunk(i32(2, 3).long(), i32(2), i32(3))
    with pytest.raises(ValueError):
        jt.hia_cache_chunk(i32(2, 3), i32(2), i32(3))
